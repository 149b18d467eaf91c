"""The draft-tree operators (rotation, attention, commit) on the GPU against the float64
oracle, on their own and as one verification step.

Tolerances, derived before the first run. A bf16 rounding is off by at most 2^-8 of the value.
Attention: the softmax weights are rounded to bf16 before the value product and the result
once at the store, so |error| <= 2^-8 |out| + 2^-8 A, A = sum_t p_t |v_t|; the fp32 scores
add a relative error of at most their own absolute error to each weight: 128 products and
sums of magnitude below 128 (2^-24 each, scaled by 1/sqrt(D)), the cap's tanh and the base-2
exponent of a bounded argument stay below 2^-11 A together. Rotation: 2^-8 |out| + 2^-20 times the
pair's size; keys one bf16 ulp, as the single-token append promises. Copies: the bits.
"""
import numpy as np
import pytest
import torch

import decode_step_attention_gb300 as dsa
from oracle import decode_ref as O
from oracle import tree as OT
from tol import check_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def f64(t):
    return t.double().cpu().numpy()


def trees(rng, B, N, empty=False):
    """Ancestor masks [B, N] (uint64) and depths of random trees."""
    mask, depth = np.zeros((B, N), np.uint64), np.zeros((B, N), np.int64)
    for b in range(B):
        for n in range(N):
            mask[b, n] = np.uint64(1 << n)
            if n and rng.random() > 0.1:
                up = int(rng.integers(max(0, n - 4), n))
                mask[b, n] |= mask[b, up]
                depth[b, n] = depth[b, up] + 1
            if empty and rng.random() < 0.3:
                mask[b, n] = 0
    return mask, depth


def attn_case(seed, lens, N, Hq, Hkv, D, T=None, nodes=None, empty=False, scale=1.0):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    T = T or max(max(lens), 1)
    rnd = lambda *s: (torch.randn(s, generator=gen) * scale).bfloat16()  # noqa: E731
    mask, depth = trees(rng, B, N, empty)
    c = dict(q=rnd(B, N, Hq, D), k_cache=rnd(B, Hkv, T, D), v_cache=rnd(B, Hkv, T, D),
             k_tree=rnd(B, Hkv, N, D), v_tree=rnd(B, Hkv, N, D))
    nodes = [N] * B if nodes is None else nodes
    for b in range(B):  # what no node may read is poison
        for name in ("k_cache", "v_cache"):
            c[name][b, :, lens[b]:] = NAN
        for name in ("k_tree", "v_tree"):
            c[name][b, :, nodes[b]:] = NAN
        c["q"][b, nodes[b]:] = NAN
    c["lens"] = torch.tensor(lens, dtype=torch.int32)
    c["n_nodes"] = torch.tensor(nodes, dtype=torch.int32)
    c["mask"] = torch.from_numpy(mask.view(np.int64))
    c["pos"] = torch.from_numpy((np.array(lens)[:, None] + depth).astype(np.int32))
    return c


TENSORS = ("q", "k_cache", "v_cache", "lens", "k_tree", "v_tree", "mask", "n_nodes", "pos")


def on_gpu(c):
    return {k: c[k].to(DEV) for k in TENSORS}


def call(g, with_pos=True, **kw):
    return dsa.gqa_tree_attn(g["q"], g["k_cache"], g["v_cache"], g["lens"], g["k_tree"],
                             g["v_tree"], g["mask"], n_nodes=g["n_nodes"],
                             pos=g["pos"] if with_pos else None, **kw)


def reference(c, **kw):
    h = {k: f64(c[k]) for k in ("q", "k_cache", "v_cache", "k_tree", "v_tree")}
    if kw.get("slopes") is not None:
        kw["slopes"] = f64(kw["slopes"])
    return OT.tree_attention(h["q"], h["k_cache"], h["v_cache"], c["lens"].numpy(), h["k_tree"],
                             h["v_tree"], c["mask"].numpy().view(np.uint64),
                             c["n_nodes"].numpy(), pos=c["pos"].numpy(), **kw)


def check(out, ref, size, what=""):
    live = ~np.isnan(ref)
    got = f64(out)
    assert np.isfinite(got[live]).all(), f"{what}: non-finite results"
    bound = 2.0 ** -8 * (np.abs(ref) + size) * 1.01 + 2.0 ** -11 * size + 1e-30
    err = np.abs(got - ref)
    bad = live & (err > bound)
    n_bad = int(bad.sum())
    assert n_bad == 0, (what, n_bad, float((err / bound)[live].max()))
    num = np.linalg.norm((got - ref)[live])
    assert num <= 4e-3 * max(np.linalg.norm(ref[live]), 1e-30), what  # the framework's RMS bound


def run(c, what="", **kw):
    g = on_gpu(c)
    ws = dsa.alloc_tree_workspace(*c["q"].shape[:3], c["k_cache"].shape[1], c["q"].shape[3],
                                  int(c["lens"].max()), kw.get("num_parts", 0))
    out = torch.full_like(g["q"], 7.0)
    okw = {k: v for k, v in kw.items() if k != "num_parts"}
    if kw.get("slopes") is not None:
        kw["slopes"] = kw["slopes"].to(DEV)
    call(g, workspace=ws, out=out, max_len=int(c["lens"].max()), **kw)
    ref, size = reference(c, **okw)
    check(out, ref, size, what)
    dead = np.isnan(ref)
    assert np.all(f64(out)[dead] == 7.0), f"{what}: a dead node's row was written"
    assert dsa.device_errors(ws) == 0, what
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", [(1, 1), (1, 8), (2, 3), (5, 4), (8, 2), (16, 8), (17, 5), (31, 7),
                                 (33, 1), (43, 6), (64, 2), (64, 8)])
def test_shapes(D, N, G):
    run(attn_case(N * G + D, [70, 1, 0, 129], N, 2 * G, 2, D), f"N={N} G={G} D={D}")


@pytest.mark.parametrize("L", [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 193, 511, 1000])
def test_lengths(L):
    run(attn_case(L, [L], 9, 4, 1, 128), f"L={L}")


@pytest.mark.parametrize("L", [100, 257, 320, 513, 577, 1000, 1217, 2000, 4100, 8600])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 1, 1, 64), (8, 16, 8, 128), (33, 8, 2, 64), (64, 8, 1, 128),
                                        (20, 8, 2, 64)])
def test_clusters_and_the_stream_by_length(L, N, Hq, Hkv, D):
    """Every number of CTAs that a sequence is shared by, with short sequences beside a long one
    (CTAs without tiles, sequences without nodes), and the stream for the same."""
    for B in (1, 4):
        c = attn_case(L + N, [L, 0, 1, 70][:B], N, Hq, Hkv, D, nodes=[N, N, max(1, N - 1), 0][:B])
        run(c, f"L={L} B={B}")
    slopes = torch.exp2(-torch.arange(1.0, Hq + 1))
    run(c, "options", softcap=25.0, slopes=slopes, window=300)
    run(c, "options", slopes=slopes)
    g = on_gpu(c)
    ws = dsa.alloc_tree_workspace(*c["q"].shape[:3], Hkv, D, L, 13)
    a = call(g, max_len=L)
    b = call(g, max_len=L, num_parts=13, workspace=ws)
    ref, size = reference(c)
    err = (a.float() - b.float()).abs().cpu().numpy()
    live = ~np.isnan(ref)
    # both within the bound of the exact result
    assert np.all(err[live] <= (2.0 ** -7 * (np.abs(ref) + size) * 1.02 + 2.0 ** -10 * size)[live])


@pytest.mark.parametrize("B,N,Hq,Hkv,D,hi", [(170, 47, 16, 4, 128, 230), (620, 3, 2, 1, 64, 1900),
                                             (40, 64, 32, 4, 64, 500)])
def test_more_short_sequences_than_the_machine_holds(B, N, Hq, Hkv, D, hi):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, hi, B)]
    nodes = [int(x) for x in rng.integers(0, N + 1, B)]
    lens[3], nodes[4] = hi, N
    run(attn_case(B, lens, N, Hq, Hkv, D, nodes=nodes, empty=True), f"B={B}")


@pytest.mark.parametrize("parts", [1, 2, 3, 7, 16, 61, 304, 1000])
def test_parts(parts):
    c = attn_case(parts, [700, 0, 5, 64, 1300, 333], 20, 8, 2, 128, nodes=[20, 20, 1, 0, 13, 7])
    run(c, f"parts={parts}", num_parts=parts)


@pytest.mark.parametrize("window", [1, 2, 5, 63, 64, 65, 200, 10000])
@pytest.mark.parametrize("parts", [0, 5])
def test_window(window, parts):
    c = attn_case(window, [300, 1, 64, 0, 777], 24, 6, 2, 64, nodes=[24, 24, 3, 24, 17])
    run(c, f"window={window}", window=window, num_parts=parts)


@pytest.mark.parametrize("gap,window", [(3, 40), (3, 3), (1, 64), (70, 200), (130, 150), (90, 20), (1, 1)])
@pytest.mark.parametrize("N,Hq,D,kw", [(3, 2, 64, {}), (20, 6, 128, {}), (64, 8, 64, {}),
                                       (9, 8, 128, {"softcap": 20.0}), (40, 6, 64, {"alibi": True})])
@pytest.mark.parametrize("parts", [0, 5])
def test_rows_behind_every_nodes_window_may_hold_anything(gap, window, N, Hq, D, kw, parts):
    """All nodes lie `gap` past the sequence's length (their parents are cached already): the first
    row any of them sees is later than for a node at the length."""
    c = attn_case(gap + window, [300, 0, 65, 20], N, Hq, 2, D, nodes=[N, N, max(1, N // 2), 1])
    c["pos"] += gap
    for b, L in enumerate((300, 0, 65, 20)):
        behind = min(L, max(0, L + gap - window + 1))
        for i, name in enumerate(("k_cache", "v_cache")):
            c[name][b, :, :behind] = (NAN, float("inf"))[(b + i) & 1]
    kw = dict(kw)
    if kw.pop("alibi", False):
        kw["slopes"] = torch.exp2(-torch.arange(1.0, Hq + 1))
    run(c, f"gap={gap} window={window}", window=window, num_parts=parts, **kw)


@pytest.mark.parametrize("softcap", [0.0, 0.5, 20.0, 50.0])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("N", [1, 13])
def test_score_options(softcap, alibi, N):
    c = attn_case(int(softcap) + N, [200, 40, 999], N, 8, 4, 128, scale=2.0)
    slopes = torch.exp2(-torch.arange(1.0, 9.0)) if alibi else None
    run(c, f"cap={softcap} alibi={alibi}", softcap=softcap, slopes=slopes)
    run(c, "with a window", softcap=softcap, slopes=slopes, window=150, scale=0.25)


@pytest.mark.parametrize("softcap", [1e-6, 200.0, 300.0, 3000.0, 1e6])
def test_caps_far_from_the_scores(softcap):
    """A cap far below the scores levels them, one far above leaves them as they are."""
    c = attn_case(21, [500, 90], 7, 8, 2, 128, scale=3.0)  # scores up to about 400
    run(c, f"cap={softcap}", softcap=softcap)
    run(c, f"cap={softcap}", softcap=softcap, scale=2.0)


@pytest.mark.parametrize("softcap", [255.0, 257.0, 1e20, 1e30])
@pytest.mark.parametrize("N", [7, 40])
def test_the_largest_caps_leave_the_scores(softcap, N):
    c = attn_case(54, [200, 64], N, 8, 2, 64)
    run(c, f"cap={softcap}", softcap=softcap)
    run(c, "no cap", softcap=softcap, slopes=torch.full((8,), 0.125))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [0.0, 20.0, 1000.0])
@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("N,G", [(8, 4), (9, 4), (16, 4), (17, 4), (64, 3)])
def test_score_options_by_rows(D, softcap, alibi, N, G):
    """Caps and biases where 4, 2 and 1 lanes share a row, over whole and ragged tiles."""
    c = attn_case(N * G + D, [400, 64, 1, 130], N, 2 * G, 2, D, nodes=[N, N - 3, N, 1], scale=2.0)
    slopes = torch.exp2(-torch.arange(1.0, 2 * G + 1)) if alibi else None
    run(c, f"cap={softcap} alibi={alibi}", softcap=softcap, slopes=slopes)
    run(c, "split", softcap=softcap, slopes=slopes, num_parts=5, window=200)


@pytest.mark.parametrize("softcap,alibi", [(30.0, False), (30.0, True), (0.0, True), (1e4, False)])
@pytest.mark.parametrize("N", [4, 12, 40])
def test_bent_scores_of_unseen_keys_change_nothing(softcap, alibi, N):
    c = attn_case(51, [90, 64], N, 8, 2, 128)
    c["mask"][:, :] = 1 << torch.arange(N, dtype=torch.int64)
    c["mask"][:, 3] |= 1 << 1
    slopes = torch.exp2(-torch.arange(1.0, 9.0)) if alibi else None
    clean = {k: v.clone() for k, v in c.items()}
    c["k_tree"][1, 0, 1, 5] = NAN  # keys 0, 2 and 3 are computed next to it
    ref, size = reference(clean, softcap=softcap, slopes=slopes)
    got = f64(call(on_gpu(c), softcap=softcap, slopes=slopes if slopes is None else slopes.to(DEV)))
    hit = np.zeros(got.shape, bool)
    hit[1, [1, 3], :4] = True
    check(torch.from_numpy(np.where(hit, ref, got)), ref, size)
    assert int(np.isfinite(got[hit]).sum()) == 0
    # a key in the cache that every node sees
    c = {k: v.clone() for k, v in clean.items()}
    c["k_cache"][0, 1, 13, 0] = NAN
    got = f64(call(on_gpu(c), softcap=softcap, slopes=slopes if slopes is None else slopes.to(DEV)))
    hit[:] = False
    hit[0, :, 4:] = True
    check(torch.from_numpy(np.where(hit, ref, got)), ref, size)
    assert int(np.isfinite(got[hit]).sum()) == 0


@pytest.mark.parametrize("softcap", [30.0, 1e4])
@pytest.mark.parametrize("N", [3, 24])
def test_scores_past_the_float_range_meet_the_cap(softcap, N):
    """Dot products that overflow fp32: their tanh is 1 or -1."""
    c = attn_case(52, [200], N, 8, 2, 128)
    c["q"][:] = 1.0
    c["k_cache"][0, :, 30] = 1e37
    c["k_cache"][0, :, 190] = 1e37
    c["k_cache"][0, :, 31] = -1e37
    c["k_tree"][0, :, 1] = -1e37
    run(c, softcap=softcap, scale=1.0)


def test_results_at_odd_16_byte_addresses():
    for N, D in ((40, 128), (40, 64), (9, 64)):
        c = attn_case(53, [100, 20], N, 8, 2, D)
        ref, size = reference(c)
        room = torch.full((c["q"].numel() + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
        out = room[8:-8].view(c["q"].shape)
        assert out.data_ptr() % 32 == 16
        call(on_gpu(c), out=out)
        check(out, ref, size)
        assert (room[:8] == 7).all() and (room[-8:] == 7).all()


def test_one_node_is_the_single_token_attention():
    """N = 1 against the framework's decode attention with the token in the cache."""
    c = attn_case(22, [700, 63, 0], 1, 8, 2, 128, T=701)
    g = on_gpu(c)
    out = call(g, max_len=700)
    kc, vc = g["k_cache"].clone(), g["v_cache"].clone()
    for b, n in enumerate((700, 63, 0)):
        kc[b, :, n], vc[b, :, n] = g["k_tree"][b, :, 0], g["v_tree"][b, :, 0]
    want = dsa.gqa_decode_attn(g["q"][:, 0].contiguous(), kc, vc, g["lens"] + 1)
    _, size = reference(c)
    err = (out[:, 0].float() - want.float()).abs().cpu().numpy()
    # both within the bound of the exact result: a bf16 rounding each, and this one's weights
    assert np.all(err <= 2.0 ** -8 * (2 * np.abs(f64(want)) + 1.1 * size[:, 0]) + 2.0 ** -10 * size[:, 0])


def test_nodes_that_see_nothing_give_zeros():
    c = attn_case(3, [0, 0, 100], 12, 4, 2, 128, empty=True)
    assert (c["mask"] == 0).any()
    run(c)
    c["mask"][:] = 0
    run(c)


def test_values_a_node_does_not_see_change_nothing():
    """NaN and inf in the key and value of one node reach only the nodes that see it."""
    for poison in (NAN, float("inf"), -float("inf")):
        for Hq, N in ((4, 12), (16, 64)):
            c = attn_case(5, [90, 64], N, Hq, 2, 128)
            c["mask"][:, :] = 1 << torch.arange(N, dtype=torch.int64)  # every node sees itself
            c["mask"][:, 3] |= 1 << 7
            clean = {k: v.clone() for k, v in c.items()}
            c["v_tree"][0, :, 7, 3:9] = poison
            c["k_tree"][1, 0, 7, 5] = NAN
            got = f64(call(on_gpu(c)))
            ref, size = reference(clean)
            hit = np.zeros(got.shape, bool)
            hit[0, [3, 7], :, 3:9] = True
            hit[1, [3, 7], :Hq // 2] = True
            check(torch.from_numpy(np.where(hit, ref, got)), ref, size)
            assert int(np.isfinite(got[hit]).sum()) == 0
    # a node nobody sees may hold anything
    c = attn_case(6, [30], 8, 4, 2, 64)
    c["mask"] &= ~(1 << 2)
    clean = {k: v.clone() for k, v in c.items()}
    c["v_tree"][:, :, 2] = NAN
    c["k_tree"][:, :, 2] = float("inf")
    ref, size = reference(clean)
    check(call(on_gpu(c)), ref, size)


def test_large_scores_and_equal_keys():
    c = attn_case(8, [400, 70], 10, 8, 2, 128, scale=8.0)  # peaked softmax, scores ~ +-700
    run(c)
    c = attn_case(9, [400, 70], 10, 8, 2, 128)
    c["k_cache"][:] = c["k_cache"][:, :, :1]
    c["k_cache"][0, :, 400:] = NAN
    c["k_cache"][1, :, 70:] = NAN
    run(c)
    # rising scores: the running maximum moves at every tile
    c = attn_case(10, [2000], 4, 4, 1, 128)
    c["q"][:] = 1.0
    c["k_cache"][0, 0] = (torch.arange(2000)[:, None] * 0.02).expand(2000, 128).bfloat16()
    run(c)
    run(c, num_parts=3)


@pytest.mark.parametrize("size", [1e3, 1e6, 1.3e8, 1e9, 1e10, 1e20, 1e35])
@pytest.mark.parametrize("N,Hq,D", [(2, 2, 64), (7, 8, 128), (24, 4, 64), (40, 8, 128)])
def test_scores_far_from_zero(size, N, Hq, D):
    """Equal scores at any size of them give the mean of the values, one larger score its value."""
    for sign in (1.0, -1.0):
        c = attn_case(N, [700, 64, 5], N, Hq, 2, D)
        live = c["k_cache"].isfinite()
        c["q"][:] = 1.0
        c["k_cache"][live] = sign * size
        c["k_tree"][:] = sign * size
        run(c, f"{sign * size}")
        run(c, "split", num_parts=7)
        c["k_cache"][0, :, 333] = 1.5 * size
        c["k_tree"][1, :, 0] = 1.5 * size
        run(c, "a peak")
        run(c, "a peak, split", num_parts=7)


def test_positions_below_the_length_count_as_the_length():
    c = attn_case(11, [100, 40], 6, 4, 2, 64)
    c["pos"][:, 2] = 3
    c["pos"][:, 4] = -5
    run(c, window=20, slopes=torch.tensor([0.5, 0.25, 0.1, 0.0]))


def test_clamped_lengths_and_counts_are_reported():
    c = attn_case(12, [40, 50], 6, 4, 2, 64, T=64)
    c["k_cache"][:] = 0.25
    c["v_cache"][:] = 0.5
    g = on_gpu(c)
    ws = dsa.alloc_tree_workspace(2, 6, 4, 2, 64, 64)
    g["lens"][0], g["lens"][1] = -3, 99
    out = call(g, workspace=ws)
    assert dsa.device_errors(ws) == dsa.DEVERR_LEN_CLAMPED
    want = dict(c, lens=torch.tensor([0, 64], dtype=torch.int32),
                pos=g["pos"].cpu())
    ref, size = reference(want)
    check(out, ref, size)
    g = on_gpu(c)
    g["n_nodes"][0], g["n_nodes"][1] = 9, -1
    ws.zero_()
    out = torch.full_like(g["q"], 7.0)
    call(g, workspace=ws, out=out)
    assert dsa.device_errors(ws) == dsa.DEVERR_TREE_CLAMPED
    assert bool((out[1] == 7.0).all()) and bool((out[0] != 7.0).any())


def test_many_sequences():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 40, 700).tolist()
    nodes = rng.integers(0, 4, 700).tolist()
    run(attn_case(13, lens, 3, 2, 1, 64, nodes=nodes))


def gpu_reference(g, slopes=None, softcap=0.0, window=0):
    """The definition in float64 torch on the GPU, a sequence at a time: (out, sum p |v|)."""
    B, N, Hq, D = g["q"].shape
    G = Hq // g["k_cache"].shape[1]
    out = torch.full(g["q"].shape, NAN, dtype=torch.float64, device=DEV)
    size = out.clone()
    node = torch.arange(N, device=DEV)
    for b in range(B):
        L, n = int(g["lens"][b]), int(g["n_nodes"][b])
        if n == 0:
            continue
        cat = lambda c, t: torch.cat([c[b, :, :L], t[b, :, :n]], 1).double()  # noqa: E731
        K = cat(g["k_cache"], g["k_tree"]).repeat_interleave(G, 0)
        V = cat(g["v_cache"], g["v_tree"]).repeat_interleave(G, 0)
        p = g["pos"][b, :n].long()
        far = p[:, None] - torch.cat([torch.arange(L, device=DEV), p])[None]
        see = torch.cat([torch.ones(n, L, dtype=torch.bool, device=DEV),
                         ((g["mask"][b, :n, None] >> node[:n]) & 1).bool()], 1)
        if window:
            see &= far < window
        z = g["q"][b, :n].double().transpose(0, 1) @ K.transpose(1, 2) / D ** 0.5
        if softcap:
            z = softcap * torch.tanh(z / softcap)
        if slopes is not None:
            z = z - slopes.double()[:, None, None] * far
        w = torch.softmax(z.masked_fill(~see, -float("inf")), -1)
        out[b, :n], size[b, :n] = (w @ V).transpose(0, 1), (w @ V.abs()).transpose(0, 1)
    return f64(out), f64(size)


@pytest.mark.parametrize("N,Hq,Hkv,D,lo,hi,kw", [
    (64, 32, 4, 128, 500, 3000, {}),                  # row tiles of 128, every SM busy
    (64, 32, 4, 128, 500, 3000, {"window": 1000}),
    (16, 32, 8, 128, 100, 4000, {"softcap": 50.0}),
    (5, 16, 4, 64, 1, 6000, {"alibi": True}),
    (1, 8, 8, 128, 1, 5000, {}),
])
def test_full_machine(N, Hq, Hkv, D, lo, hi, kw):
    """Ragged batches that keep every SM at work on many segments, several times over."""
    rng = np.random.default_rng(hi)
    B = 24
    lens = rng.integers(lo, hi, B).tolist()
    nodes = rng.integers(max(1, N // 2), N + 1, B).tolist()
    c = attn_case(17, lens, N, Hq, Hkv, D, nodes=nodes)
    g = on_gpu(c)
    kw = dict(kw)
    if kw.pop("alibi", False):
        kw["slopes"] = torch.exp2(-torch.arange(1.0, Hq + 1) / 2).to(DEV)
    ref, size = gpu_reference(g, **kw)
    first = call(g, **kw)
    check(first, ref, size)
    for _ in range(10):
        assert torch.equal(call(g, **kw), first)


def test_no_optional_arguments():
    c = attn_case(14, [77, 5], 6, 4, 2, 128)
    g = on_gpu(c)
    out = dsa.gqa_tree_attn(g["q"], g["k_cache"], g["v_cache"], g["lens"], g["k_tree"],
                            g["v_tree"], g["mask"])
    ref, size = reference(c)
    check(out, ref, size)


def test_offsets_past_32_bits():
    """The last sequence of a cache of more than 2^32 bytes and 2^31 elements."""
    B, Hkv, T, D, N = 17, 8, 131072, 128, 4
    c = attn_case(15, [200], N, 8, Hkv, D)
    kc = torch.empty(B, Hkv, T, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    kc[-1, :, :200], vc[-1, :, :200] = c["k_cache"][0].to(DEV), c["v_cache"][0].to(DEV)
    rep = lambda t: t.to(DEV).expand(B, *t.shape[1:]).contiguous()  # noqa: E731
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    lens[-1] = 200
    kt, vt, mask, q = (rep(c[k]) for k in ("k_tree", "v_tree", "mask", "q"))
    out = dsa.gqa_tree_attn(q, kc, vc, lens, kt, vt, mask, max_len=200)
    ref, size = reference(c)
    check(out[-1:], ref, size)
    path = torch.tensor([[0, 2, 3, 1]], dtype=torch.int32, device=DEV).expand(B, N).contiguous()
    count = torch.zeros_like(lens)
    count[-1] = 3
    lens[-1] = T - 3
    dsa.tree_commit(kt, vt, path, count, kc, vc, lens)
    assert torch.equal(kc[-1, :, T - 3:], kt[-1][:, [0, 2, 3]])
    assert torch.equal(vc[-1, :, T - 3:], vt[-1][:, [0, 2, 3]])


def test_same_bits_every_time_and_across_part_counts_of_one_piece():
    c = attn_case(16, [900, 30, 411], 16, 8, 2, 128)
    g = on_gpu(c)
    first = call(g)
    for _ in range(5):
        assert torch.equal(call(g), first)


def test_streams_graphs_and_a_shared_workspace():
    """On a side stream, captured and replayed, two graphs sharing one workspace in turn."""
    cs = [attn_case(20 + i, [500, 60, 0, 233], 16, 8, 2, 128) for i in range(2)]
    gs = [on_gpu(c) for c in cs]
    want = [call(g, max_len=500) for g in gs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(gs[0], max_len=500, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    ws = dsa.alloc_tree_workspace(4, 16, 8, 2, 128, 500)
    outs = [torch.zeros_like(g["q"]) for g in gs]
    graphs = []
    for g, o in zip(gs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(g, max_len=500, workspace=ws, out=o)
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    # new contents, same buffers
    gs[0]["lens"].copy_(torch.tensor([3, 499, 77, 1], dtype=torch.int32))
    gs[0]["k_cache"].nan_to_num_()
    gs[0]["v_cache"].nan_to_num_()
    eager = call(gs[0], max_len=500)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager)


def test_two_calls_at_once():
    gs = [on_gpu(attn_case(30 + i, [3000, 1500], 32, 8, 2, 128)) for i in range(2)]
    want = [call(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [call(g, stream=s) for g, s in zip(gs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_pinned_host_arguments():
    c = attn_case(40, [150, 64], 8, 4, 2, 128)
    g = on_gpu(c)
    want = call(g)
    for name in ("q", "lens", "mask", "n_nodes", "pos"):
        g[name] = c[name].pin_memory()
    got = call(g, out=torch.zeros(c["q"].shape, dtype=torch.bfloat16).pin_memory())
    torch.cuda.synchronize()
    assert torch.equal(got, want.cpu())


def test_writes_nothing_outside_its_buffers():
    c = attn_case(41, [700, 64, 3], 20, 8, 2, 128, nodes=[20, 5, 11])
    g = on_gpu(c)
    B, N, Hq, D = c["q"].shape
    for parts in (0, 7):
        n = dsa.tree_workspace_bytes(B, N, Hq, 2, D, 700, parts)
        wbuf = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
        ws = wbuf[4096:4096 + n]
        ws[:256].zero_()
        obuf = torch.full((c["q"].numel() + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
        out = obuf[2048:2048 + c["q"].numel()].view(c["q"].shape)
        call(g, workspace=ws, out=out, max_len=700, num_parts=parts)
        ref, size = reference(c)
        check(out, ref, size)
        assert bool((wbuf[:4096] == 0xA5).all()) and bool((wbuf[-4096:] == 0xA5).all())
        assert bool((obuf[:2048] == 7.0).all()) and bool((obuf[-2048:] == 7.0).all())


# -------------------------------------------------------------------- rotation ---
def rope_case(seed, B, N, Hq, Hkv, D, norm, far=1000):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen).bfloat16()  # noqa: E731
    c = dict(q=rnd(B, N, Hq, D), k_new=rnd(B, N, Hkv, D), v_new=rnd(B, N, Hkv, D),
             q_norm_w=rnd(D) if norm else None, k_norm_w=rnd(D) if norm else None,
             pos=torch.randint(0, far, (B, N), generator=gen, dtype=torch.int32),
             n_nodes=torch.randint(0, N + 1, (B,), generator=gen, dtype=torch.int32))
    return c


def run_rope(c, layout, theta=1e4, in_place=False, inv_freq=None):
    g = {k: None if v is None else v.to(DEV) for k, v in c.items()}
    B, N, Hq, D = c["q"].shape
    Hkv = c["k_new"].shape[2]
    kt = torch.full((B, Hkv, N, D), 3.0, dtype=torch.bfloat16, device=DEV)
    vt = torch.full_like(kt, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = g["q"] if in_place else torch.full_like(g["q"], 7.0)
    got = dsa.qknorm_rope_tree(g["q"], g["k_new"], g["v_new"], kt, vt, g["pos"], theta, layout,
                               g["q_norm_w"], g["k_norm_w"], n_nodes=g["n_nodes"],
                               q_out=None if in_place else q_out, error_word=err,
                               inv_freq=inv_freq)
    w = [None if c[k] is None else f64(c[k]) for k in ("q_norm_w", "k_norm_w")]
    qr, kr, vr = OT.rope_tree(f64(c["q"]), f64(c["k_new"]), f64(c["v_new"]), *w,
                              np.full(kt.shape, 3.0), np.full(vt.shape, 5.0), c["pos"].numpy(),
                              c["n_nodes"].numpy(), theta, layout, 1e-6,
                              None if inv_freq is None else inv_freq.numpy())
    live = (np.arange(N) < c["n_nodes"].numpy()[:, None]) & (c["pos"].numpy() >= 0)
    out = f64(got)
    if not in_place:
        assert np.all(out[~live] == 7.0)
    size = np.abs(qr).max(-1, keepdims=True)
    bad = np.abs(out - qr)[live] > (2.0 ** -8 * np.abs(qr) + 2.0 ** -18 * size)[live]
    assert int(bad.sum()) == 0
    check_ulp(f64(kt), kr, "tree keys")
    assert np.array_equal(f64(vt), vr)
    return int(err.item())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["neox", "interleaved"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hkv", [(1, 1, 1, 1), (3, 5, 6, 2), (2, 64, 16, 8), (9, 7, 33, 3)])
def test_rope_tree(D, layout, norm, B, N, Hq, Hkv):
    c = rope_case(B * N + D, B, N, Hq, Hkv, D, norm, far=131072)
    assert run_rope(c, layout) == 0
    assert run_rope(c, layout, in_place=True) == 0


def test_rope_tree_frequency_table_and_bad_positions():
    c = rope_case(1, 4, 6, 4, 2, 128, True)
    assert run_rope(c, "neox", inv_freq=dsa.rope_inv_freq(128, 1e6, "yarn", 8.0)) == 0
    c["n_nodes"][:] = 6
    c["pos"][1, 3] = -1
    assert run_rope(c, "neox") == dsa.DEVERR_POS_SKIPPED


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["neox", "interleaved"])
def test_rope_tree_matches_the_single_token_append(D, layout):
    """One node at a sequence's length: the bits the append writes into the cache."""
    B, Hq, Hkv, T = 200, 9, 3, 512
    c = rope_case(2, B, 1, Hq, Hkv, D, True, far=T)
    c["n_nodes"][:] = 1
    g = {k: v.to(DEV) for k, v in c.items()}
    kt = torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device=DEV)
    vt = torch.zeros_like(kt)
    q = dsa.qknorm_rope_tree(g["q"].clone(), g["k_new"], g["v_new"], kt, vt, g["pos"], 1e6, layout,
                             g["q_norm_w"], g["k_norm_w"])
    kc = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    p = g["pos"][:, 0].contiguous()
    q1 = dsa.qknorm_rope_kv_append(g["q"][:, 0].clone(), g["k_new"][:, 0].contiguous(),
                                   g["v_new"][:, 0].contiguous(), kc, vc, p, 1e6, layout,
                                   g["q_norm_w"], g["k_norm_w"])
    assert torch.equal(q[:, 0], q1)
    row = torch.arange(B, device=DEV)
    assert torch.equal(kt[:, :, 0], kc[row, :, p.long()])
    assert torch.equal(vt[:, :, 0], vc[row, :, p.long()])


@pytest.mark.parametrize("layout", ["neox", "interleaved"])
@pytest.mark.parametrize("B,N,Hq,Hkv,D", [
    # two passes of a warp over its heads; three; four; two blocks of heads per node; as many KV
    # heads as query heads, and more KV heads than one pass holds
    (3, 64, 16, 8, 128), (1, 64, 32, 32, 128), (4, 64, 32, 8, 128), (8, 64, 33, 3, 128),
    (8, 64, 24, 24, 128), (5, 62, 48, 8, 128), (8, 64, 40, 40, 128), (3, 64, 64, 32, 128),
    (6, 64, 64, 8, 128), (320, 1, 20, 20, 128), (8, 64, 16, 16, 64), (1, 64, 64, 64, 64),
    (8, 64, 48, 24, 64), (2, 64, 48, 48, 64), (8, 64, 64, 32, 64), (7, 50, 40, 40, 64)])
def test_rope_tree_several_passes(B, N, Hq, Hkv, D, layout):
    """Enough nodes and heads for a warp to turn several heads one after the other."""
    c = rope_case(N * Hq + D, B, N, Hq, Hkv, D, Hkv % 3 != 0, far=131072)
    c["n_nodes"][0] = N
    assert run_rope(c, layout) == 0
    assert run_rope(c, layout, in_place=True) == 0


@pytest.mark.parametrize("layout", ["neox", "interleaved"])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 128), (32, 8, 128), (32, 32, 128), (48, 8, 128),
                                      (64, 8, 128), (32, 16, 64), (64, 64, 64), (64, 32, 64)])
def test_rope_tree_of_many_nodes_matches_the_single_token_append(Hq, Hkv, D, layout):
    """The same bits from the forms of several passes."""
    B, T = 500, 16
    c = rope_case(Hq + D, B, 1, Hq, Hkv, D, True, far=T)
    g = {k: v.to(DEV) for k, v in c.items()}
    kt = torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device=DEV)
    vt = torch.zeros_like(kt)
    q = dsa.qknorm_rope_tree(g["q"].clone(), g["k_new"], g["v_new"], kt, vt, g["pos"], 1e6, layout,
                             g["q_norm_w"], g["k_norm_w"])
    kc = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    p = g["pos"][:, 0].contiguous()
    q1 = dsa.qknorm_rope_kv_append(g["q"][:, 0].clone(), g["k_new"][:, 0].contiguous(),
                                   g["v_new"][:, 0].contiguous(), kc, vc, p, 1e6, layout,
                                   g["q_norm_w"], g["k_norm_w"])
    row = torch.arange(B, device=DEV)
    assert torch.equal(q[:, 0], q1)
    assert torch.equal(kt[:, :, 0], kc[row, :, p.long()])
    assert torch.equal(vt[:, :, 0], vc[row, :, p.long()])


@pytest.mark.parametrize("theta", [0.5, 0.125, 2.0 ** -10])
@pytest.mark.parametrize("layout", ["neox", "interleaved"])
@pytest.mark.parametrize("D", [64, 128])
def test_rope_bases_below_one(theta, layout, D):
    """Frequencies above one radian per position, where a position is several turns."""
    assert run_rope(rope_case(D, 5, 7, 6, 2, D, True), layout, theta=theta) == 0
    B, Hq, Hkv, T = 9, 6, 2, 1000  # and the single-token append
    c = rope_case(D + 1, B, 1, Hq, Hkv, D, True, far=T)
    g = {k: v.to(DEV) for k, v in c.items()}
    kc = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    p = c["pos"][:, 0].contiguous()
    q = dsa.qknorm_rope_kv_append(g["q"][:, 0].clone(), g["k_new"][:, 0].contiguous(),
                                  g["v_new"][:, 0].contiguous(), kc, vc, p.to(DEV), theta, layout,
                                  g["q_norm_w"], g["k_norm_w"])
    turn = lambda x, w: O.qknorm_rope(f64(c[x][:, 0]), f64(c[w]), p.numpy(), theta,  # noqa: E731
                                      layout, 1e-6)
    ref = turn("q", "q_norm_w")
    assert np.all(np.abs(f64(q) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.abs(ref).max())
    check_ulp(f64(kc[torch.arange(B), :, p.long()]), turn("k_new", "k_norm_w"), "appended keys")


# ---------------------------------------------------------------------- commit ---
@pytest.mark.parametrize("B,Hkv,N,D,T", [(1, 1, 1, 64, 1), (3, 2, 5, 128, 40), (40, 8, 64, 64, 200)])
def test_commit(B, Hkv, N, D, T):
    rng = np.random.default_rng(B)
    gen = torch.Generator().manual_seed(B)
    rnd = lambda *s: torch.randn(s, generator=gen).bfloat16()  # noqa: E731
    kt, vt, kc, vc = rnd(B, Hkv, N, D), rnd(B, Hkv, N, D), rnd(B, Hkv, T, D), rnd(B, Hkv, T, D)
    path = rng.integers(0, N, (B, N))           # any order, the same node twice
    count = rng.integers(0, N + 1, B)
    lens = rng.integers(0, T + 1, B)            # some paths run past the cache's end
    i32 = lambda a: torch.from_numpy(a.astype(np.int32))  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = [t.to(DEV) for t in (kt, vt, i32(path), i32(count), kc, vc, i32(lens))]
    for _ in range(2):  # committing again changes nothing
        dsa.tree_commit(*g, error_word=err)
        k, v = OT.commit(f64(kt), f64(vt), path, count, f64(kc), f64(vc), lens)
        assert np.array_equal(f64(g[4]), k) and np.array_equal(f64(g[5]), v)
    over = bool((lens + count > T).any())
    assert int(err) == (dsa.DEVERR_POS_SKIPPED if over else 0)


def test_commit_reports_bad_nodes_and_counts():
    kt = torch.ones(2, 1, 3, 64, dtype=torch.bfloat16, device=DEV)
    kc, vc = torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16, device=DEV), None
    vc, vt = torch.zeros_like(kc), kt.clone()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsa.tree_commit(kt, vt, i32([[0, 3, -1], [0, 1, 2]]), i32([3, 9]), kc, vc, i32([0, -1]),
                    error_word=err)
    assert int(err) == dsa.DEVERR_POS_SKIPPED | dsa.DEVERR_TREE_CLAMPED
    got = kc[:, 0, :, 0].cpu().tolist()
    assert got == [[1, 0, 0, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0, 0, 0]]


# ------------------------------------------------------------- a verification step ---
def test_speculative_step_matches_sequential_decoding():
    """Drafts of several steps verified as trees and committed, against decoding the accepted
    tokens one by one with the framework's single-token operators."""
    B, N, Hq, Hkv, D, T, V, hidden = 2, 6, 4, 2, 128, 64, 512, 512
    gen = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=gen).bfloat16().to(DEV)  # noqa: E731
    w_head, table = rnd(V, Hq * D) * 0.05, [rnd(V, h, D) for h in (Hq, Hkv, Hkv)]
    lens = torch.tensor([5, 0], dtype=torch.int32, device=DEV)
    caches = [rnd(B, Hkv, T, D) for _ in range(2)]
    seq = [c.clone() for c in caches]           # the sequential side
    rng = np.random.default_rng(0)
    for step in range(4):
        mask, depth = trees(rng, B, N)
        mask[:, 1:] |= np.uint64(1)             # one root
        depth[:, 1:] = np.maximum(depth[:, 1:], 1)
        mask, depth = mask.astype(np.uint64), np.array(
            [[bin(int(m)).count("1") - 1 for m in row] for row in mask])
        tokens = torch.randint(0, V, (B, N), generator=gen).to(DEV)
        q, k, v = (t[tokens].contiguous() for t in table)
        kt, vt = torch.zeros(B, Hkv, N, D, dtype=torch.bfloat16, device=DEV), None
        vt = torch.zeros_like(kt)
        pos = (lens[:, None] + torch.from_numpy(depth).to(DEV)).int().contiguous()
        dsa.qknorm_rope_tree(q, k, v, kt, vt, pos, 1e4)
        o = dsa.gqa_tree_attn(q, *caches, lens, kt, vt,
                              torch.from_numpy(mask.view(np.int64)).to(DEV), pos=pos,
                              max_len=int(lens.max()))
        logits = dsa.linear(o.view(B * N, Hq * D), w_head)
        lp, ent, top, top_lp = dsa.token_logprobs(logits, tokens.view(-1, 1).int(), top_k=4)
        assert torch.equal(top[:, 0].long(), logits.float().argmax(1))
        assert bool((top_lp[:, 0:1] >= lp).all()) and bool((ent > 0).all())
        # accept the longest root path of node N - 1 (any path serves the comparison)
        path = np.zeros((B, N), np.int32)
        count = np.zeros(B, np.int32)
        for b in range(B):
            nodes = [j for j in range(N) if (int(mask[b, N - 1]) >> j) & 1]
            path[b, :len(nodes)], count[b] = nodes, len(nodes)
        dsa.tree_commit(kt, vt, torch.from_numpy(path).to(DEV), torch.from_numpy(count).to(DEV),
                        *caches, lens)
        # the same tokens, one at a time
        for b in range(B):
            at = lens[b:b + 1].clone()
            for i in range(int(count[b])):
                n = int(path[b, i])
                tok = tokens[b, n]
                q1, k1, v1 = (t[tok][None].contiguous() for t in table)
                kc, vc = seq[0][b:b + 1], seq[1][b:b + 1]
                dsa.qknorm_rope_kv_append(q1, k1, v1, kc, vc, at, 1e4)
                o1 = dsa.gqa_decode_attn(q1, kc, vc, at + 1)
                assert torch.allclose(o1[0].float(), o[b, n].float(), atol=2e-2, rtol=2e-2)
                at += 1
        lens += torch.from_numpy(count).to(DEV)
        for a, s in zip(caches, seq):
            assert torch.equal(a, s)


# ------------------------------------------------ all four calls, other ways to make them ---
def step_inputs(seed, B, N, Hq, Hkv, D, T, V):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen).bfloat16()  # noqa: E731
    mask, depth = trees(rng, B, N)
    lens = rng.integers(0, T - N, B)
    count = rng.integers(0, N + 1, B)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32))  # noqa: E731
    return dict(q=rnd(B, N, Hq, D), k=rnd(B, N, Hkv, D), v=rnd(B, N, Hkv, D), kc=rnd(B, Hkv, T, D),
                vc=rnd(B, Hkv, T, D), lens=i32(lens), mask=torch.from_numpy(mask.view(np.int64)),
                pos=i32(lens[:, None] + depth), nodes=i32(rng.integers(1, N + 1, B)),
                path=i32(rng.integers(0, N, (B, N))), count=i32(count),
                logits=torch.randn(B * N, V, generator=gen), ids=i32(rng.integers(0, V, (B * N, 2))),
                qw=rnd(D), kw=rnd(D))


def step(t, kt, vt, q_out, out, ws, err, T, stream=None):
    dsa.qknorm_rope_tree(t["q"], t["k"], t["v"], kt, vt, t["pos"], 1e4, q_norm_w=t["qw"],
                         k_norm_w=t["kw"], n_nodes=t["nodes"], q_out=q_out, error_word=err, stream=stream)
    dsa.gqa_tree_attn(q_out, t["kc"], t["vc"], t["lens"], kt, vt, t["mask"], n_nodes=t["nodes"],
                      pos=t["pos"], max_len=T, workspace=ws, out=out, window=40, softcap=30.0,
                      stream=stream)
    lp = dsa.token_logprobs(t["logits"], t["ids"], top_k=4, stream=stream)
    dsa.tree_commit(kt, vt, t["path"], t["count"], t["kc"], t["vc"], t["lens"], error_word=err,
                    stream=stream)
    return lp


@pytest.mark.parametrize("B,N,Hq,Hkv,D,T", [(3, 6, 8, 2, 128, 90), (40, 33, 8, 8, 64, 300)])
def test_a_step_on_a_side_stream_and_captured(B, N, Hq, Hkv, D, T):
    """The same step called on the current stream, on another, and replayed from a graph whose
    buffers then hold other inputs."""
    V = 5003
    ws = dsa.alloc_tree_workspace(B, N, Hq, Hkv, D, T)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def buffers(t):
        kt = torch.full((B, Hkv, N, D), 3.0, dtype=torch.bfloat16, device=DEV)
        q = torch.full_like(t["q"], 7.0)
        return kt, kt.clone(), q, torch.full_like(q, 9.0)

    def results(t, b, lp):
        return [x.clone() for x in (*b, t["kc"], t["vc"], *lp)]

    def on_device(seed):
        return {k: v.to(DEV) for k, v in step_inputs(seed, B, N, Hq, Hkv, D, T, V).items()}

    want = []
    for seed in (1, 2):
        t = on_device(seed)
        b = buffers(t)
        want.append(results(t, b, step(t, *b, ws, err, T)))
    side = torch.cuda.Stream()
    t = on_device(1)
    b = buffers(t)
    side.wait_stream(torch.cuda.current_stream())
    lp = step(t, *b, ws, err, T, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(results(t, b, lp), want[0]))
    t = on_device(1)
    b = buffers(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp = step(t, *b, ws, err, T)
    for seed in (2, 1, 2):
        for k, v in on_device(seed).items():
            t[k].copy_(v)
        for x, y in zip(b, buffers(t)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(results(t, b, lp), want[seed - 1])), seed
    assert int(err) == 0 and dsa.device_errors(ws) == 0


def test_a_step_with_arguments_in_pinned_host_memory():
    B, N, Hq, Hkv, D, T, V = 3, 6, 8, 2, 128, 90, 5003
    host = step_inputs(4, B, N, Hq, Hkv, D, T, V)
    got = []
    for pinned in (False, True):
        t = {k: v.to(DEV) for k, v in host.items()}
        err = torch.zeros(1, dtype=torch.int32)
        kt = torch.zeros(B, Hkv, N, D, dtype=torch.bfloat16, device=DEV)
        vt = torch.zeros_like(kt)
        q, out = torch.zeros(B, N, Hq, D, dtype=torch.bfloat16), None
        out = q.clone()
        if pinned:
            for k in t:
                if k not in ("kc", "vc", "logits"):
                    t[k] = host[k].pin_memory()
            err, q, out = err.pin_memory(), q.pin_memory(), out.pin_memory()
        else:
            err, q, out = err.to(DEV), q.to(DEV), out.to(DEV)
        ws = dsa.alloc_tree_workspace(B, N, Hq, Hkv, D, T)
        t["pos"][1, 0] = -1   # reported in the error word, wherever it lies
        lp = step(t, kt, vt, q, out, ws, err, T)
        torch.cuda.synchronize()
        assert int(err) == dsa.DEVERR_POS_SKIPPED
        got.append([x.cpu() for x in (kt, vt, q, t["kc"], t["vc"], out, *lp)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_no_sequences():
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device=DEV)  # noqa: E731
    i32, N, D = torch.int32, 4, 64
    q = dsa.qknorm_rope_tree(z(0, N, 4, D), z(0, N, 2, D), z(0, N, 2, D), z(0, 2, N, D), z(0, 2, N, D),
                             z(0, N, d=i32), 1e4)
    out = dsa.gqa_tree_attn(q, z(0, 2, 8, D), z(0, 2, 8, D), z(0, d=i32), z(0, 2, N, D),
                            z(0, 2, N, D), z(0, N, d=torch.int64))
    dsa.tree_commit(z(0, 2, N, D), z(0, 2, N, D), z(0, N, d=i32), z(0, d=i32), z(0, 2, 8, D),
                    z(0, 2, 8, D), z(0, d=i32))
    lp, ent, top, tlp = dsa.token_logprobs(z(0, 100, d=torch.float32), z(0, 3, d=i32), top_k=2)
    assert out.shape == (0, N, 4, D) and lp.shape == (0, 3) and ent.shape == (0,)
    assert top.shape == tlp.shape == (0, 2)
    lp, *_ = dsa.token_logprobs(z(2, 100, d=torch.float32), z(2, 0, d=i32))
    assert lp.shape == (2, 0)
