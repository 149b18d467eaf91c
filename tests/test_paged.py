"""The paged cache on the GPU against the float64 oracle: the append with its rotation, the
single-query attention, the gather, and a run of them as a server uses them.

Attention is held, element by element, to one bf16 step of the exact value (its rounding, twice over)
plus (2^-8 + 2^-10) sum_t p_t |v_t|: a weight is held in two e4m3 terms of 4 significant bits each,
p = hi + lo / 16 + r with |p - hi| <= 2^-4 p and |r| <= 2^-4 |p - hi|, that is 2^-8 of each; the second
term covers the scores' fp32 arithmetic. In e4m3 steps do not shrink below 2^-9, so |r| is at most half
of that over 16, 2^-14, where it is more than 2^-8 p: with the largest weight (times its value's scale) at
2^8 that is 2^-22 of the largest w = max_t p_t s_t on each code c_t, hence a third term
2^-22 w sum_t |c_t| (a value that is a zero where the large weights are, and not where the small
ones are, has nothing else to be measured by). Appended keys' and values' codes and scales have no
tolerance.
"""
import math

import numpy as np
import pytest
import torch

import decode_step_attention_gb300 as dsa
from oracle import decode_ref as O
from oracle import paged as OP
from tol import bf16_ulp, check_float, check_ulp

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def rnd(gen, *shape):
    return torch.randn(shape, generator=gen).to(BF16)


def make_cache(gen, P, Hkv, page, D, dtype, pow2=True):
    """A pool of finite values on the GPU, and the same for the oracle."""
    k, v = (torch.randn(P, Hkv, page, D, generator=gen) for _ in range(2))
    if dtype is BF16:
        k, v, ks, vs = k.to(BF16), v.to(BF16), None, None
    else:
        k, v = (64 * k).to(E4M3), (64 * v).to(E4M3)
        e = torch.randint(-9, -3, (2, P, Hkv), generator=gen).float()
        if not pow2:
            e = e + torch.rand((2, P, Hkv), generator=gen)
        ks, vs = torch.exp2(e)
    gpu = [None if t is None else t.to(DEV) for t in (k, v, ks, vs)]
    return gpu, oracle_cache(gpu)


def oracle_cache(gpu):
    return dict(zip(("k", "v", "ks", "vs"), (f64(t) for t in gpu)))


def make_table(rng, lens, page, P, width=None, first=None):
    """A table of distinct pages; entries that nothing needs are far outside the pool."""
    need = [-(-int(n) // page) for n in lens]
    skip = [0] * len(need) if first is None else [int(f) // page for f in first]
    width = max([1] + need) if width is None else width
    table = np.full((len(need), width), 0x7fffff00, dtype=np.int64)
    free = list(rng.permutation(P))
    for b, (n, s) in enumerate(zip(need, skip)):
        for j in range(s, n):
            table[b, j] = free.pop()
    return table


def check_attn(out, exact, what):
    ref, size, floor = exact
    g, err = f64(out), np.abs(f64(out) - ref)
    assert np.all(np.isfinite(g)), what
    bound = bf16_ulp(ref) + (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -22 * floor + 1e-30
    assert np.all(err <= bound), (what, float((err / bound).max()))
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(f64(out) - ref) <= 4e-3 * norm, what


def attend(q, gpu, table, lens, **kw):
    k, v, ks, vs = gpu
    B, Hq, D = q.shape
    Hkv, page = k.shape[1], k.shape[2]
    max_len = kw.pop("max_len", max(1, int(max(lens))))
    ws = kw.pop("workspace", None)
    if ws is None:
        ws = dsa.alloc_paged_workspace(B, Hq, Hkv, D, max_len, kw.get("num_parts", 0))
    out = torch.full((B, Hq, D), float("nan"), dtype=BF16, device=DEV)
    dsa.gqa_paged_attn(q, k, v, i32(table), i32(lens), k_scale=ks, v_scale=vs, max_len=max_len,
                       workspace=ws, out=out, **kw)
    torch.cuda.synchronize()
    return out, dsa.device_errors(ws)


# ---- attention ------------------------------------------------------------------------
LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 700]


@pytest.mark.parametrize("window", [0, 1, 100, 129])
@pytest.mark.parametrize("D,page,Hkv,G", [(128, 16, 2, 8), (128, 64, 1, 1), (64, 32, 3, 5),
                                          (64, 128, 2, 7), (128, 128, 1, 3), (64, 16, 1, 8)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attention(dtype, D, page, Hkv, G, window):
    gen, rng = torch.Generator().manual_seed(D + page + G), np.random.default_rng(window)
    lens = rng.permutation(LENS)
    P = sum(-(-int(n) // page) for n in lens) + 2
    gpu, ref = make_cache(gen, P, Hkv, page, D, dtype)
    first = np.maximum(0, lens - window) if window else None
    table = make_table(rng, lens, page, P, first=first)
    # what no token of a call is: NaN in rows behind the lengths, before the windows, in other pages
    real = np.zeros((P, page), dtype=bool)
    for b, n in enumerate(lens):
        for t in range(0 if first is None else first[b], n):
            real[table[b, t // page], t % page] = True
    dead = torch.from_numpy(~real).to(DEV)
    for t in gpu[:2]:
        raw = t.view(torch.uint8) if dtype is E4M3 else t.view(torch.int16)
        raw[dead[:, None].expand(P, Hkv, page)] = 0x7f if dtype is E4M3 else 0x7fff
    q = rnd(gen, len(lens), Hkv * G, D).to(DEV)
    out, err = attend(q, gpu, table, lens, window=window)
    want = OP.attention(f64(q), ref, table, lens, window=window)
    check_attn(out, want, (dtype, D, page, G, window))
    assert err == 0
    assert np.all(f64(out)[np.asarray(lens) == 0] == 0)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("parts", [0, 1, 2, 7, 152, 333])
def test_attention_any_cut(dtype, parts):
    """However the work is cut, and twice the same bits."""
    gen, rng = torch.Generator().manual_seed(5), np.random.default_rng(5)
    lens = [1500, 3, 0, 640, 129, 1, 4000]
    gpu, ref = make_cache(gen, 400, 2, 16, 128, dtype)
    table = make_table(rng, lens, 16, 400)
    q = rnd(gen, len(lens), 8, 128).to(DEV)
    ws = dsa.alloc_paged_workspace(len(lens), 8, 2, 128, 4000, parts)
    out, err = attend(q, gpu, table, lens, num_parts=parts, workspace=ws)
    want = OP.attention(f64(q), ref, table, lens)
    check_attn(out, want, (dtype, parts))
    again, err2 = attend(q, gpu, table, lens, num_parts=parts, workspace=ws)
    assert torch.equal(out, again) and err == err2 == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attention_many_sequences(dtype):
    gen, rng = torch.Generator().manual_seed(6), np.random.default_rng(6)
    lens = rng.integers(0, 300, 700)
    page, P = 32, 700 * 10
    gpu, ref = make_cache(gen, P, 1, page, 64, dtype, pow2=False)
    table = make_table(rng, lens, page, P)
    q = rnd(gen, 700, 2, 64).to(DEV)
    out, err = attend(q, gpu, table, lens)
    want = OP.attention(f64(q), ref, table, lens)
    check_attn(out, want, dtype)
    assert err == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attention_long(dtype):
    """131072 tokens, one page of them in use over and over behind others (a shared page may repeat)."""
    gen, rng = torch.Generator().manual_seed(7), np.random.default_rng(7)
    n, page, P = 131072 - 5, 128, 40
    gpu, ref = make_cache(gen, P, 2, page, 128, dtype)
    table = rng.integers(0, P, (1, 1024))
    q = rnd(gen, 1, 16, 128).to(DEV)
    out, err = attend(q, gpu, table, [n])
    want = OP.attention(f64(q), ref, table, [n])
    check_attn(out, want, dtype)
    assert err == 0


def test_attention_peaked_scores():
    """Large scores: one token takes nearly all the weight, then the tail's share matters."""
    gen, rng = torch.Generator().manual_seed(8), np.random.default_rng(8)
    lens = [3000, 3000, 700]
    for dtype in (BF16, E4M3):
        gpu, ref = make_cache(gen, 220, 1, 32, 128, dtype)
        table = make_table(rng, lens, 32, 220)
        q = (rnd(gen, 3, 4, 128) * torch.tensor([1.0, 4.0, 30.0, 0.0])[None, :, None]).to(BF16).to(DEV)
        # a sink: one row of keys along a query, its weight e^11 times the others'
        at, row = int(table[1, 0]), 5
        gpu[0][at, 0, row] = (q[1, 0].float() * (1 if dtype is BF16 else 64)).to(dtype)
        if dtype is E4M3:
            gpu[2][at, 0] = 2.0 ** -6
        ref = oracle_cache(gpu)
        out, _ = attend(q, gpu, table, lens)
        want = OP.attention(f64(q), ref, table, lens)
        check_attn(out, want, dtype)


@pytest.mark.parametrize("spread", [4, 20, 60])
def test_attention_scales_of_every_size(spread):
    """Scales of values from 2^-spread to 2^spread side by side in a tile; queries far apart in size."""
    gen, rng = torch.Generator().manual_seed(spread), np.random.default_rng(spread)
    lens = [16, 130, 1000, 77]
    gpu, _ = make_cache(gen, 90, 2, 16, 128, E4M3)
    gpu[3].copy_(torch.exp2(torch.randint(-spread, spread + 1, gpu[3].shape, generator=gen).float()))
    table = make_table(rng, lens, 16, 90)
    ref = oracle_cache(gpu)
    q = rnd(gen, 4, 8, 128)
    q[:, 1] *= 2.0 ** -20
    q[:, 2, ::2] *= 2.0 ** -9
    q[:, 3] = 0
    q = q.to(DEV)
    out, _ = attend(q, gpu, table, lens)
    want = OP.attention(f64(q), ref, table, lens)
    check_attn(out, want, spread)


def test_attention_of_8192_sequences():
    """The most sequences of a call, none or one token each: a value or zeros."""
    gen, rng = torch.Generator().manual_seed(32), np.random.default_rng(32)
    for dtype in (BF16, E4M3):
        lens = rng.integers(0, 2, 8192)
        gpu, ref = make_cache(gen, 64, 1, 16, 64, dtype)
        table = rng.integers(0, 64, (8192, 1))
        q = rnd(gen, 8192, 2, 64).to(DEV)
        out, err = attend(q, gpu, table, lens)
        v = ref["v"][table[:, 0], 0, 0] * (1 if dtype is BF16 else ref["vs"][table[:, 0], 0][:, None])
        want = np.where(lens[:, None, None] > 0, v[:, None, :], 0.0)
        check_ulp(f64(out), np.broadcast_to(want, (8192, 2, 64)), "one token", 0.5)
        assert err == 0


def test_one_workspace_for_calls_of_every_shape():
    """One workspace, of the largest call's size, for calls of other shapes and types in between."""
    rng = np.random.default_rng(33)
    shapes = [(1, 8, 8, 128, 16, [5000]), (7, 8, 1, 64, 32, [900, 3, 70, 0, 128, 1500, 2]),
              (2, 14, 2, 64, 128, [4000, 129]), (40, 4, 4, 128, 64, list(range(1, 400, 10)))]
    ws = torch.zeros(max(dsa.paged_workspace_bytes(B, Hq, Hkv, D, max(n))
                         for B, Hq, Hkv, D, _, n in shapes), dtype=torch.uint8, device=DEV)
    for turn in range(2):
        for dtype in (E4M3, BF16):
            for B, Hq, Hkv, D, page, lens in shapes:
                gen = torch.Generator().manual_seed(turn + Hq)
                P = sum(-(-n // page) for n in lens)
                gpu, ref = make_cache(gen, P, Hkv, page, D, dtype)
                table = make_table(rng, lens, page, P)
                q = rnd(gen, B, Hq, D).to(DEV)
                out, err = attend(q, gpu, table, lens, workspace=ws)
                check_attn(out, OP.attention(f64(q), ref, table, lens), (turn, dtype, B, Hq))
                assert err == 0


def test_attention_scale_argument():
    gen, rng = torch.Generator().manual_seed(9), np.random.default_rng(9)
    for dtype in (BF16, E4M3):
        gpu, ref = make_cache(gen, 30, 2, 32, 64, dtype)
        lens = [300, 200]
        table = make_table(rng, lens, 32, 30)
        q = rnd(gen, 2, 6, 64).to(DEV)
        for scale in (1.0, 0.01, -1.0):
            out, _ = attend(q, gpu, table, lens, scale=scale)
            want = OP.attention(f64(q), ref, table, lens, scale=max(scale, 0))
            check_attn(out, want, (dtype, scale))


def test_attention_far_pages():
    """Pages behind 2^32 bytes of the pool."""
    gen, rng = torch.Generator().manual_seed(10), np.random.default_rng(10)
    for dtype in (BF16, E4M3):
        size = 2 if dtype is BF16 else 1
        P, Hkv, page, D = (9 << 29) // (16 * 64 * 128 * size), 16, 64, 128   # 4.5 GiB each
        small, _ = make_cache(gen, 12, Hkv, page, D, dtype)
        k, v = (torch.empty(P, Hkv, page, D, dtype=dtype, device=DEV) for _ in range(2))
        at = torch.cat([torch.arange(P - 10, P), torch.tensor([0, P // 2])])
        raw = torch.uint8 if dtype is E4M3 else torch.int16
        for big, t in ((k, small[0]), (v, small[1])):
            big.view(raw)[at.to(DEV)] = t.view(raw)
        ks = vs = None
        if dtype is E4M3:
            ks, vs = (torch.ones(P, Hkv, device=DEV) for _ in range(2))
            ks[at.to(DEV)], vs[at.to(DEV)] = small[2], small[3]
        pick = rng.permutation(12)
        table, local = at.numpy()[pick][None], pick[None]
        q = rnd(gen, 1, 16, D).to(DEV)
        out, err = attend(q, (k, v, ks, vs), table, [12 * 64 - 7])
        want = OP.attention(f64(q), oracle_cache(small), local, [12 * 64 - 7])
        check_attn(out, want, dtype)
        ko, vo = (torch.zeros(1, Hkv, 40, D, dtype=BF16, device=DEV) for _ in range(2))
        dsa.paged_gather(k, v, i32(table), i32([12 * 64]), ko, vo, ks, vs, start=i32([12 * 64 - 40]))
        K, V, _ = OP.tokens(oracle_cache(small), local, 0, 12 * 64 - 40, 12 * 64)
        check_ulp(f64(ko[0]), K, "far gather", 0.5)
        check_ulp(f64(vo[0]), V, "far gather", 0.5)
        # the append into the last page
        new = rnd(gen, 1, Hkv, D).to(DEV)
        dsa.qknorm_rope_paged_append(q, new, new, k, v, i32([[P - 1]]), i32([3]), 1e4, k_scale=ks,
                                     v_scale=vs, rot_dim=0)
        dsa.paged_gather(k, v, i32([[P - 1]]), i32([4]), ko, vo, ks, vs, start=i32([3]))
        got = f64(vo[0, :, 0])
        assert np.all(np.abs(got - f64(new[0])) <= np.abs(f64(new[0])) * 2.0 ** -4 + 1e-2)
        del k, v, big


def test_attention_flags_bad_pages_and_lengths():
    gen, rng = torch.Generator().manual_seed(11), np.random.default_rng(11)
    for dtype in (BF16, E4M3):
        gpu, ref = make_cache(gen, 40, 2, 16, 128, dtype)
        lens = [200, 90, 33]
        table = make_table(rng, lens, 16, 40)
        table[0, 2], table[0, 11], table[1, 5], table[2, :3] = -1, 40, -(1 << 31), (1 << 31) - 1
        q = rnd(gen, 3, 4, 128).to(DEV)
        out, err = attend(q, gpu, table, lens)
        want = OP.attention(f64(q), ref, table, lens)
        check_attn(out, want, dtype)
        assert err == dsa.DEVERR_PAGE_SKIPPED and bool((out[2] == 0).all())
        table = make_table(rng, lens, 16, 40)
        out, err = attend(q, gpu, table, [300, -5, 33], max_len=200)
        want = OP.attention(f64(q), ref, table, [200, 0, 33])
        check_attn(out, want, dtype)
        assert err == dsa.DEVERR_LEN_CLAMPED


def test_attention_nan_stays_with_its_sequence_and_head():
    gen, rng = torch.Generator().manual_seed(12), np.random.default_rng(12)
    for dtype in (BF16, E4M3):
        gpu, _ = make_cache(gen, 40, 2, 16, 64, dtype)
        lens = [200, 150]
        table = make_table(rng, lens, 16, 40)
        raw = gpu[1].view(torch.uint8 if dtype is E4M3 else torch.int16)
        raw[int(table[0, 3]), 1, 4, 9] = 0x7f if dtype is E4M3 else 0x7fc0
        q = rnd(gen, 2, 8, 64).to(DEV)
        out, _ = attend(q, gpu, table, lens)
        bad = torch.isnan(out)
        assert bool(bad[0, 4:, 9].all())
        bad[0, 4:, 9] = False
        assert not bool(bad.any())


# ---- append -----------------------------------------------------------------------------
def run_append(gen, rng, dtype, D, page, Hq, Hkv, layout, rot, norm, start, new, theta=1e4, big=1.0,
               single=False, packed=False, in_place=False, pow2=True):
    B, n = len(start), int(np.sum(new))
    total = np.asarray(start) + np.asarray(new)
    P = int(sum(-(-int(t) // page) for t in total)) + 3
    gpu, ref = make_cache(gen, P, Hkv, page, D, dtype, pow2)
    table = make_table(rng, total, page, P)
    if packed:
        qkv = rnd(gen, n, (Hq + 2 * Hkv) * D).to(DEV)
        q = qkv[:, :Hq * D].view(n, Hq, D)
        k, v = (qkv[:, (Hq + i * Hkv) * D:(Hq + (i + 1) * Hkv) * D].view(n, Hkv, D) for i in (0, 1))
    else:
        q, k, v = (rnd(gen, n, h, D).to(DEV) for h in (Hq, Hkv, Hkv))
    size = torch.exp2(torch.randint(-3, 4, (n, 1, 1), generator=gen).float()).to(DEV) * big
    k.mul_(size.to(BF16))
    v.mul_(size.flip(0).to(BF16))
    w = (1 + 0.1 * rnd(gen, 2, D).float()).to(BF16).to(DEV) if norm else None
    cu = None if single else np.concatenate([[0], np.cumsum(new)])
    args = (f64(q), f64(k), f64(v), ref, table, start, cu, theta, layout, rot)
    q_want, c_want = OP.append(*args, *((f64(w[0]), f64(w[1])) if norm else (None, None)))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = None if in_place else torch.zeros(n, Hq, D, dtype=BF16, device=DEV)
    got = dsa.qknorm_rope_paged_append(
        q, k, v, gpu[0], gpu[1], i32(table), i32(start), theta, cu_new=None if single else i32(cu),
        k_scale=gpu[2], v_scale=gpu[3], layout=layout, rot_dim=rot, q_norm_w=w[0] if norm else None,
        k_norm_w=w[1] if norm else None, q_out=q_out, error_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    what = (dtype, D, page, layout, rot, norm)
    check_float(f64(got), q_want, f"q {what}")
    if dtype is BF16:
        check_ulp(f64(gpu[0]), c_want["k"], f"keys {what}")
    else:
        assert np.array_equal(f64(gpu[2]), c_want["ks"]), what
        assert np.array_equal(f64(gpu[3]), c_want["vs"]), what
        assert np.array_equal(f64(gpu[0]), c_want["k"]), (what, int((f64(gpu[0]) != c_want["k"]).sum()))
    assert np.array_equal(f64(gpu[1]), c_want["v"]), what
    return gpu, table


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("layout", ["neox", "interleaved"])
@pytest.mark.parametrize("D,page,rot", [(128, 16, 128), (128, 64, 32), (64, 32, 64), (64, 128, 16),
                                        (128, 128, 112), (64, 16, 0)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_append_prompts(dtype, D, page, rot, layout, norm):
    """Ragged prompts, from a page's first row and from inside one, with sequences that get nothing."""
    gen = torch.Generator().manual_seed(D + page + rot)
    run_append(gen, np.random.default_rng(rot), dtype, D, page, 6, 2, layout, rot, norm,
               [0, 5, 130, 16, 7, 127, 0, 300], [200, 1, 0, 31, page, 3, 1, 2 * page + 1])


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("layout", ["neox", "interleaved"])
@pytest.mark.parametrize("D,page,Hq,Hkv,rot", [(128, 16, 16, 8, 128), (64, 64, 7, 7, 32),
                                               (128, 32, 5, 1, 16), (64, 128, 40, 20, 64)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_append_tokens(dtype, D, page, Hq, Hkv, rot, layout, norm):
    """One token per sequence, at every place of a page."""
    gen, rng = torch.Generator().manual_seed(Hq), np.random.default_rng(Hq)
    start = np.concatenate([[0, 1, page - 1, page, page + 1, 2 * page - 1], rng.integers(0, 400, 31)])
    run_append(gen, rng, dtype, D, page, Hq, Hkv, layout, rot, norm, start, np.ones(37, dtype=int),
               single=True)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n", [1, 2, 3, 33, 300])
def test_append_token_batches(dtype, n):
    gen, rng = torch.Generator().manual_seed(n), np.random.default_rng(n)
    run_append(gen, rng, dtype, 128, 16, 4, 2, "neox", 128, True, rng.integers(0, 40, n),
               np.ones(n, dtype=int), single=True)


@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** -12])
def test_append_scales_grow_or_stay(big):
    """New tokens far above and far below what a page holds; scales of any value in the page before."""
    for pow2 in (True, False):
        gen, rng = torch.Generator().manual_seed(3), np.random.default_rng(3)
        run_append(gen, rng, E4M3, 128, 64, 2, 2, "neox", 64, False, [10, 63, 0, 40, 7],
                   [20, 70, 3, 1, 60], big=big, pow2=pow2)
        run_append(gen, rng, E4M3, 64, 32, 2, 2, "interleaved", 64, True, [10, 31, 0, 20, 7],
                   np.ones(5, dtype=int), big=big, single=True, pow2=pow2)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_append_far_positions(dtype):
    gen, rng = torch.Generator().manual_seed(4), np.random.default_rng(4)
    run_append(gen, rng, dtype, 128, 128, 4, 1, "neox", 128, True, [130944, 70001], [129, 1],
               theta=1e6)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("single", [True, False])
def test_append_from_a_packed_projection(dtype, single):
    """q, k and v as column blocks of [n, (Hq + 2 Hkv) D], q rotated where it lies."""
    gen, rng = torch.Generator().manual_seed(13), np.random.default_rng(13)
    new = np.ones(9, dtype=int) if single else [40, 1, 90]
    run_append(gen, rng, dtype, 64, 16, 6, 3, "interleaved", 32, True, rng.integers(0, 50, len(new)), new,
               single=single, packed=True, in_place=True)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("page", [16, 64])
def test_append_mixed_batch(dtype, page):
    """Prompts among many sequences that get one token each, or none: more than 32 sequences."""
    gen, rng = torch.Generator().manual_seed(34), np.random.default_rng(34)
    new = rng.choice([0, 1, 1, 1, 2, 9], 90)
    new[[7, 50]] = 150, 33
    run_append(gen, rng, dtype, 64, page, 4, 2, "neox", 64, True, rng.integers(0, 200, 90), new)


def test_append_where_every_element_is_on_a_border():
    """Keys that lie halfway between two codes, which only their exact value settles (ties to even),
    in more places than the kernel's lists hold: nothing turns (frequencies of zero), as prompts and as
    single tokens, with scales that stay and scales that grow."""
    gen, rng = torch.Generator().manual_seed(35), np.random.default_rng(35)
    for layout in ("neox", "interleaved"):
        for D, page, single in ((128, 64, False), (64, 128, False), (128, 16, True), (128, 128, False)):
            start = [0, 5, 70] if not single else [0, 3, 17, 40]
            new = [page + 9, 40, 3] if not single else [1, 1, 1, 1]
            B, n = len(start), sum(new)
            P = 3 * B * (2 + 160 // page)
            gpu, ref = make_cache(gen, P, 2, page, D, E4M3)
            table = make_table(rng, np.add(start, new), page, P)
            steps = torch.randint(8, 16, (n, 2, D), generator=gen).float() + 0.5
            k = (steps * torch.exp2(torch.randint(-5, 3, (n, 2, D), generator=gen).float())).to(BF16).to(DEV)
            q, v = rnd(gen, n, 4, D).to(DEV), rnd(gen, n, 2, D).to(DEV)
            cu = None if single else np.concatenate([[0], np.cumsum(new)])
            inv = torch.zeros(D // 2, dtype=torch.float64)
            _, c = OP.append(f64(q), f64(k), f64(v), ref, table, start, cu, 1e4, layout, D,
                             inv_freq=inv.numpy())
            dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], i32(table), i32(start), 1e4,
                                         cu_new=None if single else i32(cu), k_scale=gpu[2],
                                         v_scale=gpu[3], layout=layout, inv_freq=inv)
            assert np.array_equal(f64(gpu[2]), c["ks"])
            assert np.array_equal(f64(gpu[0]), c["k"]), (layout, D, page, single)
            assert np.array_equal(f64(gpu[1]), c["v"])


@pytest.mark.parametrize("n", [3, 40])
def test_append_where_every_rotation_cancels(n):
    """bf16 keys of equal pairs turned by an eighth of a turn: the first of each pair nearly vanishes, and
    is within one step of what it is."""
    gen, rng = torch.Generator().manual_seed(36), np.random.default_rng(36)
    for layout in ("neox", "interleaved"):
        gpu, ref = make_cache(gen, 100, 3, 16, 128, BF16)
        start = np.full(n, 999)
        table = rng.permutation(100)[:n][:, None].repeat(63, 1)
        q = rnd(gen, n, 6, 128).to(DEV)
        half = rnd(gen, n, 3, 64)
        k = (torch.cat([half, half], -1) if layout == "neox" else half.repeat_interleave(2, -1)).to(DEV)
        inv = torch.full((64,), math.pi / 4 / 999, dtype=torch.float64)
        _, c = OP.append(f64(q), f64(k), f64(k), ref, table, start, None, 1e4, layout, 128,
                         inv_freq=inv.numpy())
        dsa.qknorm_rope_paged_append(q, k, k.clone(), gpu[0], gpu[1], i32(table), i32(start), 1e4,
                                     layout=layout, inv_freq=inv)
        # (what nearly vanishes goes by the angle's own rounding, 2^-64 of a turn a position)
        small = 2.0 ** -64 * 2 * math.pi * 999 * 8
        g, want = f64(gpu[0]), c["k"]
        assert np.all(np.abs(g - want) <= bf16_ulp(want) + small), np.abs(g - want).max()


@pytest.mark.parametrize("n", [31, 32, 33, 64, 65, 129])
@pytest.mark.parametrize("D", [64, 128])
def test_append_at_the_edges_of_a_block(D, n):
    """As many tokens as a block has rows, and one less and one more."""
    for norm, rot in ((False, D), (True, D // 2)):
        for layout in ("neox", "interleaved"):
            gen, rng = torch.Generator().manual_seed(n), np.random.default_rng(n)
            run_append(gen, rng, BF16, D, 32, 9, 3, layout, rot, norm, rng.integers(0, 90, n),
                       np.ones(n, dtype=int), single=True, in_place=norm)
            for dtype in (BF16, E4M3):
                run_append(gen, rng, dtype, D, 64, 9, 3, layout, rot, norm, [7], [n], in_place=norm)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_append_many_heads(dtype):
    gen, rng = torch.Generator().manual_seed(41), np.random.default_rng(41)
    run_append(gen, rng, dtype, 64, 128, 66, 33, "neox", 64, False, [100, 0], [180, 90])
    run_append(gen, rng, dtype, 128, 128, 33, 33, "interleaved", 128, True, [100, 0], [180, 90])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_append_prompts_from_host_memory(dtype):
    gen, rng = torch.Generator().manual_seed(42), np.random.default_rng(42)
    start, new = [3, 0], [100, 61]
    gpu, ref = make_cache(gen, 12, 2, 16, 64, dtype)
    table = make_table(rng, np.add(start, new), 16, 12)
    q, k, v = (rnd(gen, 161, h, 64).pin_memory() for h in (6, 2, 2))
    cu = torch.tensor([0, 100, 161], dtype=torch.int32).pin_memory()
    at = torch.tensor(start, dtype=torch.int32).pin_memory()
    q_want, c = OP.append(f64(q), f64(k), f64(v), ref, table, start, [0, 100, 161], 1e4, "neox", 64)
    dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], i32(table), at, 1e4, cu_new=cu,
                                 k_scale=gpu[2], v_scale=gpu[3])
    torch.cuda.synchronize()
    check_float(f64(q), q_want, "host q")
    check_ulp(f64(gpu[0]), c["k"], "keys")
    assert np.array_equal(f64(gpu[1]), c["v"])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_append_prompts_captured(dtype):
    """A captured append, replayed with other sequences, starts and tables of the same number of tokens."""
    gen, rng = torch.Generator().manual_seed(43), np.random.default_rng(43)
    n, B, P, page = 150, 4, 80, 32
    gpu, _ = make_cache(gen, P, 2, page, 128, dtype)
    q, k, v = (torch.zeros(n, h, 128, dtype=BF16, device=DEV) for h in (4, 2, 2))
    q_out = torch.zeros_like(q)
    table = torch.zeros(B, 16, dtype=torch.int32, device=DEV)
    start, cu = (torch.zeros(m, dtype=torch.int32, device=DEV) for m in (B, B + 1))

    def body():
        dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], table, start, 1e4, cu_new=cu,
                                     k_scale=gpu[2], v_scale=gpu[3], q_out=q_out)

    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for _ in range(3):
        s, ends = rng.integers(0, 200, B), np.sort(rng.integers(0, n + 1, B - 1))
        c = np.concatenate([[0], ends, [n]])
        t = make_table(rng, s + np.diff(c), page, P, width=16)
        table.copy_(i32(t)), start.copy_(i32(s)), cu.copy_(i32(c))
        for x in (q, k, v):
            x.copy_(rnd(gen, *x.shape))
        q_want, want = OP.append(f64(q), f64(k), f64(v), oracle_cache(gpu), t, s, c, 1e4, "neox", 128)
        graph.replay()
        torch.cuda.synchronize()
        check_float(f64(q_out), q_want, "captured q")
        check_ulp(f64(gpu[0]), want["k"], "captured keys")
        assert np.array_equal(f64(gpu[1]), want["v"])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_nothing_beside_the_buffers_is_written(dtype):
    """Guard bytes around all that append, attention and gather write."""
    gen, rng = torch.Generator().manual_seed(44), np.random.default_rng(44)
    B, Hq, Hkv, D, page, rows = 3, 6, 2, 64, 16, 90
    start, new = np.array([40, 0, 15]), np.array([33, 70, 1])
    lens, n = start + new, int(new.sum())
    P = int(sum(-(-m // page) for m in lens))
    gpu, ref = make_cache(gen, P, Hkv, page, D, dtype)
    table = make_table(rng, lens, page, P)
    pad, spaces = 4096, []

    def guarded(like):
        raw = torch.full((2 * pad + like.numel() * like.element_size(),), 0x5a, dtype=torch.uint8,
                         device=DEV)
        t = raw[pad:-pad].view(like.dtype).view(like.shape)
        t.copy_(like)
        spaces.append(raw)
        return t

    k, v, ks, vs = (None if t is None else guarded(t) for t in gpu)
    q_out = guarded(torch.zeros(n, Hq, D, dtype=BF16, device=DEV))
    out = guarded(torch.zeros(B, Hq, D, dtype=BF16, device=DEV))
    ko, vo = (guarded(torch.zeros(B, Hkv, rows, D, dtype=BF16, device=DEV)) for _ in range(2))
    ws = guarded(dsa.alloc_paged_workspace(B, Hq, Hkv, D, int(lens.max())))
    err = guarded(torch.zeros(1, dtype=torch.int32, device=DEV))
    q, kn, vn = (rnd(gen, n, h, D).to(DEV) for h in (Hq, Hkv, Hkv))
    cu = np.concatenate([[0], np.cumsum(new)])
    dsa.qknorm_rope_paged_append(q, kn, vn, k, v, i32(table), i32(start), 1e4, cu_new=i32(cu), k_scale=ks,
                                 v_scale=vs, q_out=q_out, error_word=err)
    last = q_out[torch.from_numpy(cu[1:] - 1).to(DEV)].contiguous()
    dsa.gqa_paged_attn(last, k, v, i32(table), i32(lens), ks, vs, max_len=int(lens.max()), workspace=ws,
                       out=out)
    dsa.paged_gather(k, v, i32(table), i32(lens), ko, vo, ks, vs, error_word=err)
    torch.cuda.synchronize()
    for raw in spaces:
        assert bool((raw[:pad] == 0x5a).all()) and bool((raw[-pad:] == 0x5a).all())
    _, want = OP.append(f64(q), f64(kn), f64(vn), ref, table, start, cu, 1e4, "neox", D)
    check_ulp(f64(k), want["k"], "keys")
    assert np.array_equal(f64(v), want["v"]) and int(err) == 0
    check_attn(out, OP.attention(f64(last), oracle_cache((k, v, ks, vs)), table, lens), "out")


def test_append_values_without_a_scale():
    """Zeros, infinities and NaN: a page of zeros has the smallest scale, and neither of the others
    sets one."""
    k, v, ks, vs = dsa.alloc_paged_cache(4, 16, 1, 64)
    x = torch.zeros(3, 1, 64, dtype=BF16, device=DEV)
    table = i32([[1], [2], [3]])
    x[1, 0, 0], x[1, 0, 1], x[1, 0, 2], x[1, 0, 3] = float("inf"), float("nan"), -1.0, float("-inf")
    x[2, 0, 5] = 3.3e38
    dsa.qknorm_rope_paged_append(x.clone(), x, x, k, v, table, i32([0, 0, 0]), 1e4, k_scale=ks, v_scale=vs,
                                 rot_dim=0)
    for s in (ks, vs):
        assert s[1, 0] == 2.0 ** -64 and s[2, 0] == 2.0 ** -8 and s[3, 0] == 2.0 ** 120
    for p in (k, v):
        row = p.float()[2, 0, 0]
        assert row[0] == 448 and torch.isnan(row[1]) and row[2] == -256 and row[3] == -448
        assert bool((p.float()[1] == 0).all())


def test_append_skips_what_has_no_place():
    gen, rng = torch.Generator().manual_seed(14), np.random.default_rng(14)
    for dtype in (BF16, E4M3):
        for single in (True, False):
            gpu, ref = make_cache(gen, 6, 2, 16, 64, dtype)
            table = np.array([[0, 6], [1, -7], [2, 3], [4, 5]])
            start = [16, 20, -1, 32]   # a bad page, a bad page, a bad start, behind the table
            new = [1, 1, 1, 1] if single else [2, 1, 3, 5]
            n = sum(new)
            cu = np.concatenate([[0], np.cumsum(new)])
            q, k, v = (rnd(gen, n, h, 64).to(DEV) for h in (4, 2, 2))
            before = [t if t is None else t.clone() for t in gpu]
            q_want, _ = OP.append(f64(q), f64(k), f64(v), ref, table, start, cu, 1e4, "neox", 64)
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], i32(table), i32(start), 1e4,
                                         cu_new=None if single else i32(cu), k_scale=gpu[2],
                                         v_scale=gpu[3], error_word=err)
            assert int(err) == dsa.DEVERR_PAGE_SKIPPED | dsa.DEVERR_POS_SKIPPED
            check_float(f64(q), q_want, "q of skipped tokens")
            for a, b in zip(gpu, before):
                assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_leaves_tokens_of_no_sequence():
    gen = torch.Generator().manual_seed(15)
    for dtype in (BF16, E4M3):
        gpu, _ = make_cache(gen, 6, 2, 16, 64, dtype)
        q, k, v = (rnd(gen, 20, h, 64).to(DEV) for h in (4, 2, 2))
        q0, before = q.clone(), [t if t is None else t.clone() for t in gpu]
        dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], i32([[1, 2], [3, 4]]), i32([0, 9]), 1e4,
                                     cu_new=i32([3, 8, 12]), k_scale=gpu[2], v_scale=gpu[3])
        assert torch.equal(q[:3], q0[:3]) and torch.equal(q[12:], q0[12:])
        assert not torch.equal(q[3:12], q0[3:12])
        for a, b in zip(gpu[:2], before):
            rows = (a.view(torch.uint8) != b.view(torch.uint8)).flatten(3).any(-1).any(1)
            assert bool(rows[1, :5].all()) and bool(rows[3, 9:13].all())
            rows[1, :5] = rows[3, 9:13] = False
            if dtype is E4M3:
                rows[3, :9] = False  # (what the page held, under a scale that may have grown)
            assert not bool(rows.any())


def test_append_frequency_table():
    gen, rng = torch.Generator().manual_seed(16), np.random.default_rng(16)
    gpu, ref = make_cache(gen, 9, 2, 16, 128, E4M3)
    table = make_table(rng, [40, 30], 16, 9)
    q, k, v = (rnd(gen, 30, h, 128).to(DEV) for h in (4, 2, 2))
    inv = dsa.rope_inv_freq(64, 1e4, "yarn", 4.0, 4096)
    q_want, c = OP.append(f64(q), f64(k), f64(v), ref, table, [20, 20], [0, 20, 30], 1e4, "neox", 64,
                          inv_freq=inv.numpy())
    dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], i32(table), i32([20, 20]), 0.0,
                                 cu_new=i32([0, 20, 30]), k_scale=gpu[2], v_scale=gpu[3], rot_dim=64,
                                 inv_freq=inv)
    check_float(f64(q), q_want, "q with a table")
    assert np.array_equal(f64(gpu[0]), c["k"]) and np.array_equal(f64(gpu[1]), c["v"])


# ---- gather -------------------------------------------------------------------------------
@pytest.mark.parametrize("D,page,Hkv", [(128, 16, 2), (64, 128, 3), (128, 64, 1), (64, 32, 2)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_gather(dtype, D, page, Hkv):
    gen, rng = torch.Generator().manual_seed(D + page), np.random.default_rng(page)
    lens = np.array([0, 1, page, page + 1, 500, 63, 64, 130])
    start = np.array([0, 0, 3, page, 123, 62, 70, 0])
    P = int(sum(-(-n // page) for n in lens)) + 1
    gpu, ref = make_cache(gen, P, Hkv, page, D, dtype, pow2=False)
    table = make_table(rng, lens, page, P)
    for st, rows in ((None, 500), (start, 377)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ko, vo = (torch.full((8, Hkv, rows, D), 7.0, dtype=BF16, device=DEV) for _ in range(2))
        dsa.paged_gather(gpu[0], gpu[1], i32(table), i32(lens), ko, vo, gpu[2], gpu[3],
                         start=None if st is None else i32(st), error_word=err)
        for b, n in enumerate(lens):
            s = 0 if st is None else int(st[b])
            K, V, _ = OP.tokens(ref, table, b, min(s, n), int(n))
            for out, want in ((ko, K), (vo, V)):
                check_ulp(f64(out[b, :, :max(0, n - s)]), want, "gather", 0.5)
                assert bool((out[b, :, max(0, n - s):] == 7).all())
        assert int(err) == 0


@pytest.mark.parametrize("B,rows", [(20, 600), (64, 1000)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_gather_into_long_caches(dtype, B, rows):
    """Room for many more rows than there are tokens, in more blocks than the SMs hold."""
    gen, rng = torch.Generator().manual_seed(B), np.random.default_rng(B)
    lens = rng.integers(0, 330, B)
    P = int(sum(-(-n // 32) for n in lens))
    gpu, ref = make_cache(gen, P, 8, 32, 64, dtype, pow2=False)
    table = make_table(rng, lens, 32, P)
    ko, vo = (torch.full((B, 8, rows, 64), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    dsa.paged_gather(gpu[0], gpu[1], i32(table), i32(lens), ko, vo, gpu[2], gpu[3])
    for b, n in enumerate(lens):
        K, V, _ = OP.tokens(ref, table, b, 0, int(n))
        for out, want in ((ko, K), (vo, V)):
            check_ulp(f64(out[b, :, :n]), want, "gather", 0.5)
            assert bool((out[b, :, n:] == 7).all())


def test_gather_flags():
    gen = torch.Generator().manual_seed(1)
    gpu, ref = make_cache(gen, 5, 1, 16, 64, BF16)
    table = np.array([[0, 9, 2], [3, 4, -1]])
    ko, vo = (torch.full((2, 1, 20, 64), 7.0, dtype=BF16, device=DEV) for _ in range(2))

    def call(lens, start):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        dsa.paged_gather(gpu[0], gpu[1], i32(table), i32(lens), ko, vo, start=i32(start), error_word=err)
        return int(err)
    assert call([20, 20], [0, 0]) == dsa.DEVERR_PAGE_SKIPPED
    assert bool((ko[0, :, 16:] == 7).all()) and np.array_equal(f64(ko[1, 0, :16]), ref["k"][3, 0])
    assert call([16, 32], [0, 0]) == dsa.DEVERR_LEN_CLAMPED     # more than `rows` tokens
    assert call([16, 1 << 30], [0, 30]) == dsa.DEVERR_LEN_CLAMPED | dsa.DEVERR_PAGE_SKIPPED
    assert call([16, -3], [0, 0]) == dsa.DEVERR_LEN_CLAMPED
    assert call([4, 0], [-2, 5]) == dsa.DEVERR_POS_SKIPPED


# ---- together -----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,D,page", [(E4M3, 128, 16), (BF16, 64, 32), (E4M3, 64, 128)])
def test_a_server_run(dtype, D, page):
    """Prompts of several lengths, then tokens one by one: append and attention against the oracle
    fed with the cache as it stands, and the contiguous calls over a gathered cache beside them."""
    gen, rng = torch.Generator().manual_seed(21), np.random.default_rng(21)
    B, Hq, Hkv, steps = 4, 8, 2, 20
    new = np.array([70, 1, 33, 128])
    P = B * -(-(128 + steps) // page)
    k, v, ks, vs = dsa.alloc_paged_cache(P, page, Hkv, D, dtype)
    table = rng.permutation(P).reshape(B, -1)
    t_gpu, start = i32(table), torch.zeros(B, dtype=torch.int32, device=DEV)
    n = int(new.sum())
    q, kn, vn = (rnd(gen, n, h, D).to(DEV) for h in (Hq, Hkv, Hkv))
    dsa.qknorm_rope_paged_append(q, kn, vn, k, v, t_gpu, start, 1e4, k_scale=ks, v_scale=vs,
                                 cu_new=i32(np.concatenate([[0], np.cumsum(new)])))
    start += i32(new)
    ws = dsa.alloc_paged_workspace(B, Hq, Hkv, D, 128 + steps)
    hidden = 256
    norm_w = rnd(gen, hidden).to(DEV)
    for step in range(steps):
        lens = start + 1
        x, res = (rnd(gen, B, hidden).to(DEV) for _ in range(2))
        res0 = res.clone()
        q, kn, vn = (rnd(gen, B, h, D).to(DEV) for h in (Hq, Hkv, Hkv))
        q0, y, out = q.clone(), torch.empty_like(x), torch.empty_like(q)
        before = oracle_cache((k, v, ks, vs))
        dsa.paged_decode_step(x, res, norm_w, y, q, kn, vn, k, v, t_gpu, start, lens, out, ws, 1e4,
                              k_scale=ks, v_scale=vs, max_len=128 + steps)
        torch.cuda.synchronize()
        after = oracle_cache((k, v, ks, vs))
        q_want, want = OP.append(f64(q0), f64(kn), f64(vn), before, table, f64(start).astype(int), None, 1e4,
                                 "neox", D)
        check_float(f64(q), q_want, "step q")
        if dtype is E4M3:
            for name in want:
                assert np.array_equal(after[name], want[name]), (step, name)
        else:
            check_ulp(after["k"], want["k"], "step keys")
        ref = OP.attention(f64(q), after, table, f64(lens).astype(int))
        check_attn(out, ref, step)
        y_ref, s_ref = O.rmsnorm_residual(f64(x), f64(res0), f64(norm_w), 1e-6)
        check_float(f64(y), y_ref, "step y")
        check_ulp(f64(res), s_ref, "step residual")
        if step % 10 == 9:  # the calls over contiguous caches
            kc, vc = (torch.zeros(B, Hkv, 128 + steps, D, dtype=BF16, device=DEV) for _ in range(2))
            dsa.paged_gather(k, v, t_gpu, lens, kc, vc, ks, vs)
            flat = dsa.gqa_decode_attn(q, kc, vc, lens)
            check_attn(flat, ref, ("contiguous", step))
        start += 1
    assert dsa.device_errors(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_captured_and_on_another_stream(dtype):
    """A step on a side stream, captured and replayed with other tokens, lengths and tables; two
    graphs that share a workspace, one after the other."""
    gen, rng = torch.Generator().manual_seed(22), np.random.default_rng(22)
    B, Hq, Hkv, D, page, P, top = 3, 8, 2, 128, 16, 150, 700
    gpu, _ = make_cache(gen, P, Hkv, page, D, dtype)
    k, v, ks, vs = gpu
    table = torch.zeros(B, -(-top // page), dtype=torch.int32, device=DEV)
    pos, lens = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    q, kn, vn = (torch.zeros(B, h, D, dtype=BF16, device=DEV) for h in (Hq, Hkv, Hkv))
    out = torch.zeros_like(q)
    ws = dsa.alloc_paged_workspace(B, Hq, Hkv, D, top)

    def body():
        dsa.qknorm_rope_paged_append(q, kn, vn, k, v, table, pos, 1e4, k_scale=ks, v_scale=vs)
        dsa.gqa_paged_attn(q, k, v, table, lens, ks, vs, max_len=top, workspace=ws, out=out)

    def fill():
        n = rng.integers(1, top, B)
        t = make_table(rng, n, page, P, width=table.shape[1])
        table.copy_(i32(t)), lens.copy_(i32(n)), pos.copy_(i32(n - 1))
        for x in (q, kn, vn):
            x.copy_(rnd(gen, *x.shape))
        return n, t

    def check(n, t, what):
        torch.cuda.synchronize()
        ref = OP.attention(f64(q), oracle_cache(gpu), t, n)
        check_attn(out, ref, what)

    side = torch.cuda.Stream()
    n, t = fill()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    check(n, t, "side stream")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            body()
        graphs.append(g)
    for i in range(4):
        n, t = fill()
        graphs[i % 2].replay()
        check(n, t, ("replay", i))
    # the stream argument
    n, t = fill()
    side.wait_stream(torch.cuda.current_stream())
    dsa.qknorm_rope_paged_append(q, kn, vn, k, v, table, pos, 1e4, k_scale=ks, v_scale=vs, stream=side)
    got = dsa.gqa_paged_attn(q, k, v, table, lens, ks, vs, max_len=top, stream=side)
    side.synchronize()
    out.copy_(got)
    check(n, t, "stream argument")
    assert dsa.device_errors(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_pages_beyond_32_bits(dtype):
    """A pool of more than 2^32 bytes per tensor, whose last pages are in use."""
    gen, rng = torch.Generator().manual_seed(45), np.random.default_rng(45)
    Hkv, page, D, used = 8, 128, 128, 20
    P = 2 ** 32 // (Hkv * page * D * (2 if dtype is BF16 else 1)) + used
    if torch.cuda.mem_get_info()[0] < 16 * 2 ** 30:
        pytest.skip("needs 10 GB of device memory")
    k, v, ks, vs = dsa.alloc_paged_cache(P, page, Hkv, D, dtype)
    start, new = np.array([200, 0, 126]), np.array([70, 300, 1])
    lens, n = start + new, int(new.sum())
    near = make_table(rng, lens, page, used)
    far = np.where(near < used, near + P - used, near)
    gpu, ref = make_cache(gen, used, Hkv, page, D, dtype)
    for t, x in zip((k, v, ks, vs), gpu):
        if t is not None:
            t[P - used:].copy_(x)
    q, kn, vn = (rnd(gen, n, h, D).to(DEV) for h in (16, Hkv, Hkv))
    cu = np.concatenate([[0], np.cumsum(new)])
    q_want, want = OP.append(f64(q), f64(kn), f64(vn), ref, near, start, cu, 1e4, "neox", D)
    dsa.qknorm_rope_paged_append(q, kn, vn, k, v, i32(far), i32(start), 1e4, cu_new=i32(cu), k_scale=ks,
                                 v_scale=vs)
    check_float(f64(q), q_want, "q")
    check_ulp(f64(k[P - used:]), want["k"], "far keys")
    assert np.array_equal(f64(v[P - used:]), want["v"])
    last = q[torch.from_numpy(cu[1:] - 1).to(DEV)].contiguous()
    out, err = attend(last, (k, v, ks, vs), far, lens)
    now = oracle_cache([None if t is None else t[P - used:] for t in (k, v, ks, vs)])
    check_attn(out, OP.attention(f64(last), now, near, lens), "far pages")
    rows = int(lens.max())
    ko, vo = (torch.zeros(3, Hkv, rows, D, dtype=BF16, device=DEV) for _ in range(2))
    dsa.paged_gather(k, v, i32(far), i32(lens), ko, vo, ks, vs)
    for b, m in enumerate(lens):
        K, V, _ = OP.tokens(now, near, b, 0, int(m))
        check_ulp(f64(ko[b, :, :m]), K, "gather", 0.5)
        check_ulp(f64(vo[b, :, :m]), V, "gather", 0.5)
    assert err == 0
    for t in (k, v):  # (page 0, where a wrapped offset would land)
        assert not bool(t[:used].view(torch.uint8 if dtype is E4M3 else torch.int16).any())


@pytest.mark.parametrize("single", [True, False])
def test_captured_appends_leave_their_scales(single):
    """Scales and codes of a captured append in e4m3, replayed on other tokens, starts and tables; scales of
    other pages stay."""
    gen, rng = torch.Generator().manual_seed(47), np.random.default_rng(47)
    B, P, page = 5, 80, 16
    n = B if single else 130
    gpu, _ = make_cache(gen, P, 2, page, 128, E4M3)
    q, k, v = (torch.zeros(n, h, 128, dtype=BF16, device=DEV) for h in (4, 2, 2))
    q_out = torch.zeros_like(q)
    table = torch.zeros(B, 16, dtype=torch.int32, device=DEV)
    start, cu = (torch.zeros(m, dtype=torch.int32, device=DEV) for m in (B, B + 1))

    def body():
        dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], table, start, 1e4,
                                     cu_new=None if single else cu, k_scale=gpu[2], v_scale=gpu[3],
                                     q_out=q_out)

    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for turn in range(4):
        s = rng.integers(0, 100, B)
        c = np.arange(B + 1) if single else np.concatenate([[0], np.sort(rng.integers(0, n + 1, B - 1)), [n]])
        t = make_table(rng, s + np.diff(c), page, P, width=16)
        table.copy_(i32(t)), start.copy_(i32(s)), cu.copy_(i32(c))
        for x in (q, k, v):  # (larger from turn to turn: scales grow)
            x.copy_((rnd(gen, *x.shape).float() * 4.0 ** (turn - 1)).to(BF16))
        _, want = OP.append(f64(q), f64(k), f64(v), oracle_cache(gpu), t, s, c, 1e4, "neox", 128)
        graph.replay()
        torch.cuda.synchronize()
        for got, name in zip(gpu, ("k", "v", "ks", "vs")):
            assert np.array_equal(f64(got), want[name]), (turn, name)


@pytest.mark.parametrize("single", [True, False])
def test_scales_of_pages_beyond_32_bits(single):
    """A pool of more than 2^32 bytes per tensor: the scales and codes of its last pages after an append, and
    nothing of the others'."""
    gen, rng = torch.Generator().manual_seed(48), np.random.default_rng(48)
    Hkv, page, D, used = 8, 64, 128, 20
    P = 2 ** 32 // (Hkv * page * D) + used
    if torch.cuda.mem_get_info()[0] < 16 * 2 ** 30:
        pytest.skip("needs 10 GB of device memory")
    k, v, ks, vs = dsa.alloc_paged_cache(P, page, Hkv, D, E4M3)
    start = np.array([200, 0, 127, 63])
    new = np.ones(4, dtype=int) if single else np.array([70, 300, 1, 2])
    lens, n = start + new, int(new.sum())
    near = make_table(rng, lens, page, used)
    far = np.where(near < used, near + P - used, near)
    gpu, ref = make_cache(gen, used, Hkv, page, D, E4M3)
    for t, x in zip((k, v, ks, vs), gpu):
        t[P - used:].copy_(x)
    q, kn, vn = (rnd(gen, n, h, D).to(DEV) for h in (16, Hkv, Hkv))
    cu = None if single else np.concatenate([[0], np.cumsum(new)])
    _, want = OP.append(f64(q), f64(kn), f64(vn), ref, near, start, cu, 1e4, "neox", D)
    dsa.qknorm_rope_paged_append(q, kn, vn, k, v, i32(far), i32(start), 1e4,
                                 cu_new=None if single else i32(cu), k_scale=ks, v_scale=vs)
    for got, name in zip((k, v, ks, vs), ("k", "v", "ks", "vs")):
        assert np.array_equal(f64(got[P - used:]), want[name]), name
    assert bool((ks[:P - used] == 1).all()) and bool((vs[:P - used] == 1).all())
    for t in (k, v):
        assert not bool(t[:used].view(torch.uint8).any())


def test_attention_of_no_tokens_at_all():
    gen = torch.Generator().manual_seed(46)
    gpu, _ = make_cache(gen, 2, 2, 16, 64, E4M3)
    q = rnd(gen, 3, 4, 64).to(DEV)
    for max_len in (0, 16):
        out, err = attend(q, gpu, np.full((3, 1), -1), [0, 0, 0], max_len=max_len)
        assert not bool(out.any()) and err == 0


def test_host_memory():
    """Queries, lengths and outputs in pinned host memory."""
    gen, rng = torch.Generator().manual_seed(23), np.random.default_rng(23)
    lens = [100, 37]
    gpu, ref = make_cache(gen, 12, 2, 16, 64, E4M3)
    table = make_table(rng, lens, 16, 12)
    q, k, v = (rnd(gen, 2, h, 64).pin_memory() for h in (6, 2, 2))
    start = torch.tensor([99, 36], dtype=torch.int32).pin_memory()
    n = torch.tensor(lens, dtype=torch.int32).pin_memory()
    out = torch.zeros(2, 6, 64, dtype=BF16).pin_memory()
    q_want, c = OP.append(f64(q), f64(k), f64(v), ref, table, [99, 36], None, 1e4, "neox", 64)
    t = i32(table)
    dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], t, start, 1e4, k_scale=gpu[2], v_scale=gpu[3])
    dsa.gqa_paged_attn(q, gpu[0], gpu[1], t, n, gpu[2], gpu[3], out=out)
    torch.cuda.synchronize()
    check_float(f64(q), q_want, "host q")
    assert np.array_equal(f64(gpu[0]), c["k"])
    want = OP.attention(f64(q), oracle_cache(gpu), table, lens)
    check_attn(out, want, "host out")


def test_two_streams_with_workspaces_of_their_own():
    gen, rng = torch.Generator().manual_seed(24), np.random.default_rng(24)
    lens = [5000, 3000]
    gpu, ref = make_cache(gen, 260, 2, 32, 128, E4M3)
    table = make_table(rng, lens, 32, 260)
    qs = [rnd(gen, 2, 16, 128).to(DEV) for _ in range(2)]
    t, n = i32(table), i32(lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [dsa.alloc_paged_workspace(2, 16, 2, 128, 5000) for _ in range(2)]
    outs = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, s, ws, out in zip(qs, streams, spaces, outs):
            dsa.gqa_paged_attn(q, gpu[0], gpu[1], t, n, gpu[2], gpu[3], max_len=5000, workspace=ws,
                               out=out, stream=s)
    torch.cuda.synchronize()
    for q, out in zip(qs, outs):
        want = OP.attention(f64(q), ref, table, lens)
        check_attn(out, want, "two streams")


def equal_keys(gen, value, P, Hkv, page, D, dtype, pow2=True):
    """A pool whose keys are all `value` (at most four significant bits), in e4m3 under scales that
    differ from page to page, and values under scales of any size."""
    gpu, _ = make_cache(gen, P, Hkv, page, D, dtype, pow2)
    if dtype is BF16:
        gpu[0].fill_(value)
    else:
        e = math.frexp(value)[1]
        up = torch.randint(0, 6, (P, Hkv), generator=gen).to(DEV)
        code = torch.exp2(up.float()) * (value * 2.0 ** -e)
        gpu[0].copy_(code[:, :, None, None].expand(gpu[0].shape).to(E4M3))
        gpu[2].copy_(torch.exp2((e - up).float()))
    return gpu


@pytest.mark.parametrize("e", [9, 12, 16, 20, 24, 25, 27, 28, 30, 66, 116])
@pytest.mark.parametrize("dtype,D,page,G", [(E4M3, 128, 16, 4), (E4M3, 128, 64, 7), (E4M3, 64, 32, 8),
                                            (E4M3, 64, 128, 2), (BF16, 128, 32, 3), (BF16, 64, 16, 8)])
def test_attention_scores_far_from_zero(dtype, D, page, G, e):
    """Equal scores of some 2^e give the mean of the values, one larger score its value, one smaller
    score nothing, whatever the scales of keys and values and however the tokens are cut."""
    gen, rng = torch.Generator().manual_seed(e + D + G), np.random.default_rng(e)
    lens = [700, 64, 5, 1300]
    P = sum(-(-n // page) for n in lens)
    for sign in (1.0, -1.0):
        for pow2 in (True, False):
            size = sign * 1.25 * 2.0 ** e
            gpu = equal_keys(gen, size, P, 2, page, D, dtype, pow2)
            table = make_table(rng, lens, page, P)
            q = torch.ones(4, 2 * G, D, dtype=BF16, device=DEV)
            q[:, 1::3] = 0.5
            for peak in (False, True):
                if peak:  # 1.5 times as far: a page's row
                    at, row = int(table[0, 333 // page]), 333 % page
                    gpu[0][at, :, row] = (1.5 * gpu[0][at, :, row].float()).to(dtype)
                want = OP.attention(f64(q), oracle_cache(gpu), table, lens)
                for parts in (0, 7):
                    out, err = attend(q, gpu, table, lens, num_parts=parts)
                    check_attn(out, want, (dtype, D, page, G, size, pow2, peak, parts))
                    assert err == 0


@pytest.mark.parametrize("dtype,D,page,G", [(E4M3, 128, 16, 4), (E4M3, 64, 32, 8), (BF16, 128, 32, 3),
                                            (BF16, 64, 16, 8)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("falls", [False, True])
def test_attention_scores_that_grow(falls, sign, dtype, D, page, G):
    """Scores that double from page to page, from small to far ones and back: a call's partials and sums
    lie at bases far apart."""
    gen, rng = torch.Generator().manual_seed(D + G), np.random.default_rng(D)
    lens = [70 * page - 3, 9 * page, 1, 40 * page]
    P = sum(-(-n // page) for n in lens)
    gpu, _ = make_cache(gen, P, 2, page, D, dtype)
    table = make_table(rng, lens, page, P)
    for b, n in enumerate(lens):
        pages = [int(at) for at in table[b, :-(-n // page)]]
        for j, at in enumerate(pages[::-1] if falls else pages):
            if dtype is BF16:
                gpu[0][at] = sign * 1.5 * 2.0 ** (j - 8)
            else:
                gpu[0][at] = torch.full((2, page, D), sign * 1.5 * 2.0 ** (j % 5), device=DEV).to(E4M3)
                gpu[2][at] = 2.0 ** (j - 8 - j % 5)
    q = torch.ones(4, 2 * G, D, dtype=BF16, device=DEV)
    q[:, ::2] = -0.75
    want = OP.attention(f64(q), oracle_cache(gpu), table, lens)
    for parts in (0, 1, 40):
        out, err = attend(q, gpu, table, lens, num_parts=parts)
        check_attn(out, want, (dtype, D, page, G, sign, falls, parts))
        assert err == 0


@pytest.mark.parametrize("e", [-120, -100, -60, 60, 100, 110, 117, 120])
@pytest.mark.parametrize("dtype,D", [(E4M3, 128), (E4M3, 64), (BF16, 128)])
def test_attention_queries_of_every_size(dtype, D, e):
    """Queries of some 2^e over keys of some 2^-e."""
    gen, rng = torch.Generator().manual_seed(D), np.random.default_rng(0)
    lens = [300, 40]
    gpu, _ = make_cache(gen, 30, 2, 16, D, dtype)
    table = make_table(rng, lens, 16, 30)
    if dtype is BF16:
        gpu[0].copy_((gpu[0].float() * 2.0 ** -e).to(BF16))
    else:
        gpu[2].copy_(torch.full((30, 2), 2.0 ** (-e - 6)))
    q = (rnd(gen, 2, 8, D).double() * 2.0 ** e).to(BF16).to(DEV)
    assert bool(q.isfinite().all())
    out, err = attend(q, gpu, table, lens)
    check_attn(out, OP.attention(f64(q), oracle_cache(gpu), table, lens), (dtype, D, e))
    assert err == 0


@pytest.mark.parametrize("lo,hi", [(-64, -64), (-64, 36), (19, 119), (119, 119)])
def test_attention_values_at_the_ends_of_their_scales(lo, hi):
    """Values' scales from one end of their range to the other, short and long contexts."""
    gen, rng = torch.Generator().manual_seed(hi), np.random.default_rng(0)
    for D, G, n in ((128, 2, 131072), (64, 8, 3000), (128, 5, 17)):
        gpu, _ = make_cache(gen, 40, 1, 32, D, E4M3)
        gpu[3].copy_(torch.exp2(torch.randint(lo, hi + 1, gpu[3].shape, generator=gen).float()))
        gpu[3][0], gpu[3][1] = 2.0 ** lo, 2.0 ** hi
        table = rng.integers(0, 40, (1, -(-n // 32)))
        q = rnd(gen, 1, G, D).to(DEV)
        out, err = attend(q, gpu, table, [n])
        check_attn(out, OP.attention(f64(q), oracle_cache(gpu), table, [n]), (lo, hi, D, n))
        assert err == 0


@pytest.mark.parametrize("dtype,D,page,G", [(E4M3, 128, 16, 3), (E4M3, 64, 32, 7), (BF16, 128, 64, 8)])
def test_attention_far_and_common_scores_side_by_side(dtype, D, page, G):
    """Heads of far, equal scores beside heads of common ones in the same tiles, with a window, a page that
    does not exist, sequences of common scores before and after, and what no token is not a number."""
    gen, rng = torch.Generator().manual_seed(G), np.random.default_rng(G)
    lens, window, e = [300, 700, 0, 200, 33], 450, 40
    P = sum(-(-n // page) for n in lens)
    gpu, _ = make_cache(gen, P, 2, page, D, dtype)
    table = make_table(rng, lens, page, P)
    for at in table[1, :-(-lens[1] // page)]:  # the second sequence: half of a key's elements the same
        if dtype is BF16:
            gpu[0][int(at)] = (gpu[0][int(at)].float() * 2.0 ** e).to(BF16)
            gpu[0][int(at), ..., :D // 2] = 1.25 * 2.0 ** e
        else:
            j = int(rng.integers(0, 5))
            gpu[0][int(at), ..., :D // 2] = torch.full((2, page, D // 2), 1.25 * 2.0 ** j, device=DEV).to(E4M3)
            gpu[2][int(at)] = 2.0 ** (e - j)
    table[1, 9] = -7
    if lens[1] % page:
        raw = gpu[1].view(torch.uint8 if dtype is E4M3 else torch.int16)
        raw[int(table[1, -(-lens[1] // page) - 1]), :, lens[1] % page:] = 0x7f if dtype is E4M3 else 0x7fff
    q = rnd(gen, 5, 2 * G, D).double()
    q[1, ::2, D // 2:] = 0                      # far scores, alike over the tokens
    q[1, 1::2, :D // 2] = 0
    q[1, 1::2] *= 2.0 ** -(e + (0 if dtype is BF16 else 6))
    q = q.to(BF16).to(DEV)
    for parts in (0, 3):
        out, err = attend(q, gpu, table, lens, window=window, num_parts=parts)
        want = OP.attention(f64(q), oracle_cache(gpu), table, lens, window=window)
        check_attn(out, want, (dtype, D, page, G, parts))
        # (a page wholly before the window is not looked up)
        assert err == (dsa.DEVERR_PAGE_SKIPPED if 10 * page > lens[1] - window else 0)


@pytest.mark.parametrize("dtype,D,page,G", [(E4M3, 128, 32, 3), (E4M3, 64, 64, 7), (BF16, 128, 16, 8),
                                            (BF16, 64, 128, 4)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_far_scores_amid_common_ones(sign, dtype, D, page, G):
    """Two pages of far, equal scores amid a sequence of common ones, in every third head 0 instead, and
    common sequences on either side: all of it in one piece, in few, and in many."""
    gen, rng = torch.Generator().manual_seed(D + G), np.random.default_rng(D + G)
    lens = [333, 1500, 40, 900]
    P = sum(-(-n // page) for n in lens)
    gpu, _ = make_cache(gen, P, 2, page, D, dtype)
    gpu[0][..., 0] = 0
    table = make_table(rng, lens, page, P)
    for at in table[1, 640 // page:640 // page + 2]:
        gpu[0][int(at)] = 0
        gpu[0][int(at), ..., 0] = sign * 1.5 * (1.0 if dtype is E4M3 else 2.0 ** 40)
        if dtype is E4M3:
            gpu[2][int(at)] = 2.0 ** 40
    q = rnd(gen, 4, 2 * G, D)
    q[..., 0] = 1
    q[:, ::3, 0] = 0
    q = q.to(BF16).to(DEV)
    want = OP.attention(f64(q), oracle_cache(gpu), table, lens)
    for parts in (0, 1, 3, 40):
        out, err = attend(q, gpu, table, lens, num_parts=parts)
        check_attn(out, want, (dtype, D, page, G, sign, parts))
        assert err == 0


@pytest.mark.parametrize("falls", [False, True])
def test_attention_far_scores_a_step_apart(falls):
    """Scores of 2^27.3 (in powers of two) that rise or fall by 16, one step of fp32 there, every 32
    tokens: a weight of 2^-16 stays one. The softmax scale is ln 2, so that a score is its q . k."""
    gen, rng = torch.Generator().manual_seed(3), np.random.default_rng(3)
    lens = [640, 130, 40]
    gpu, _ = make_cache(gen, 60, 1, 16, 128, BF16)
    table = make_table(rng, lens, 16, 60)
    for b, n in enumerate(lens):
        for t in range(n):
            j = t // 32 % 5
            row = gpu[0][int(table[b, t // 16]), 0, t % 16]
            row[:127] = 1.25 * 2.0 ** 20
            row[127] = 256.0 * (4 - j if falls else j)
    q = torch.ones(3, 4, 128, dtype=BF16, device=DEV)
    q[..., 127] = 2.0 ** -4
    ln2 = float(np.float32(math.log(2.0)))
    want = OP.attention(f64(q), oracle_cache(gpu), table, lens, scale=ln2)
    for parts in (0, 1, 7):
        out, err = attend(q, gpu, table, lens, num_parts=parts, scale=ln2)
        check_attn(out, want, (falls, parts))
        assert err == 0


@pytest.mark.parametrize("dtype,D", [(E4M3, 64), (E4M3, 128), (BF16, 64)])
def test_the_longest_contexts(dtype, D):
    """Sequences of nearly 2^31 tokens (a table may name a page over and over): a token appended, a window
    and the last rows of them, beside a short sequence."""
    gen, rng = torch.Generator().manual_seed(D), np.random.default_rng(D)
    page, M, P, window = 64, 2 ** 25 - 1, 40, 300
    lens = np.array([M * page, 90, M * page - 1, 1])
    gpu, ref = make_cache(gen, P, 2, page, D, dtype)
    table = np.full((4, M), 39, dtype=np.int32)
    table[:, -8:] = np.arange(32).reshape(4, 8)
    table[1, :2], table[3, 0] = [32, 33], 34
    t, start, n = i32(table), i32(lens - 1), i32(lens)
    q, k, v = (rnd(gen, 4, h, D).to(DEV) for h in (8, 2, 2))
    q_want, want = OP.append(f64(q), f64(k), f64(v), ref, table, lens - 1, None, 1e4, "neox", D)
    dsa.qknorm_rope_paged_append(q, k, v, gpu[0], gpu[1], t, start, 1e4, k_scale=gpu[2], v_scale=gpu[3])
    check_float(f64(q), q_want, "q")
    check_ulp(f64(gpu[0]), want["k"], "keys")
    now = oracle_cache(gpu)
    for parts in (0, 5):
        ws = dsa.alloc_paged_workspace(4, 8, 2, D, M * page, parts)
        out = torch.full_like(q, float("nan"))
        dsa.gqa_paged_attn(q, gpu[0], gpu[1], t, n, gpu[2], gpu[3], workspace=ws, out=out, window=window,
                           num_parts=parts)
        torch.cuda.synchronize()
        assert dsa.device_errors(ws) == 0
        check_attn(out, OP.attention(f64(q), now, table, lens, window=window), (dtype, D, parts))
    first = np.maximum(lens - 200, 0)
    ko, vo = (torch.zeros(4, 2, 200, D, dtype=BF16, device=DEV) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsa.paged_gather(gpu[0], gpu[1], t, n, ko, vo, gpu[2], gpu[3], start=i32(first), error_word=err)
    assert int(err) == 0
    for b, (lo, m) in enumerate(zip(first, lens)):
        K, V, _ = OP.tokens(now, table, b, int(lo), int(m))
        check_ulp(f64(ko[b, :, :m - lo]), K, "gather", 0.5)
        check_ulp(f64(vo[b, :, :m - lo]), V, "gather", 0.5)
