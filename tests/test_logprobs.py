"""token_logprobs on the GPU against the float64 oracle.

Tolerance, derived before the first run: log probabilities are (z - M) / T - ln S in fp32.
The sum S of V <= 262144 exponentials is off by at most 2^-24 per addition on the longest
chain (below 600: each thread's own terms, then the reductions) and 2^-21 from the
exponentials, so ln S by less than 4e-5; the other terms by a few 2^-24 of their size. The
entropy's second sum errs in the same proportion to its value, at most ln V.
"""
import numpy as np
import pytest
import torch

import decode_step_attention_gb300 as dsa
from oracle import tree as OT

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(z, ids, K, T=1.0, vocab=None):
    lp, ent, top, tlp = dsa.token_logprobs(z.to(DEV), ids.to(DEV), top_k=K, temperature=T,
                                           vocab=vocab)
    V = vocab or z.shape[1]
    rows = z[:, :V].double().numpy()
    for b in range(z.shape[0]):
        rlp, rent, rtop, rtlp = OT.logprobs(rows[b], ids[b].tolist(), K, T)
        for got, ref in ((lp[b], rlp), (tlp[b] if K else None, rtlp)):
            if got is None:
                continue
            got = got.double().cpu().numpy()
            inf = np.isneginf(ref)
            assert np.array_equal(np.isneginf(got), inf)
            assert np.all(np.abs(got - ref)[~inf] <= 4e-5 + 2.0 ** -21 * np.abs(ref[~inf]))
        assert abs(float(ent[b]) - rent) <= 4e-5 * (1 + rent)
        if K:
            assert top[b].tolist() == list(rtop), (b, K)
    return lp, ent, top, tlp


def make(seed, B, V, kind="peaked", dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn(B, V, generator=gen) * 2
    if kind == "peaked":
        at = torch.randint(0, V, (B, 16), generator=gen)
        z.scatter_add_(1, at, 8 + 3 * torch.randn(B, 16, generator=gen))
    elif kind == "flat":
        z[:] = 0.5
    elif kind == "rising":
        z = torch.arange(V).float().expand(B, V) * (8.0 / V)
    elif kind == "steps":                       # many equal values
        z = torch.randint(-3, 4, (B, V), generator=gen).float()
    elif kind == "masked":
        z[torch.rand(B, V, generator=gen) < 0.9] = -float("inf")
        z[:, V // 2] = 1.0
    elif kind == "huge":
        z *= 1e4
    return z.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 100, 1000, 4096, 4097, 16384, 32767, 50257, 65537,
                               131072, 151936, 262143, 262144])
def test_sizes(V, dtype):
    z = make(V, 3, V, dtype=dtype)
    gen = torch.Generator().manual_seed(V)
    ids = torch.randint(0, V, (3, 5), generator=gen, dtype=torch.int32)
    run(z, ids, min(20, V))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["flat", "rising", "steps", "masked", "huge"])
@pytest.mark.parametrize("V", [50, 5000, 40000, 262144])
def test_rows(kind, V, dtype):
    z = make(1, 2, V, kind, dtype)
    ids = torch.tensor([[0, V - 1, V // 2], [1, V // 3, 2]], dtype=torch.int32)
    for K in (0, 1, 5, 32):
        run(z, ids, K)


@pytest.mark.parametrize("T", [0.1, 0.7, 1.0, 3.0])
def test_temperature(T):
    run(make(2, 4, 3001), torch.arange(8, dtype=torch.int32).view(4, 2), 8, T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,ld", [(50257, 50304), (999, 1001), (5, 130), (32001, 32003)])
def test_padded_rows(V, ld, dtype):
    z = make(3, 5, ld, dtype=dtype)
    z[:, V:] = float("nan")
    run(z, torch.full((5, 1), V - 1, dtype=torch.int32), 3, vocab=V)


@pytest.mark.parametrize("B", [1, 2, 77, 300, 2500])
def test_many_rows(B):
    run(make(B, B, 777), torch.randint(0, 777, (B, 3), dtype=torch.int32), 4)


def test_ids_outside_and_repeated():
    z = make(4, 2, 100)
    lp, *_ = run(z, torch.tensor([[-1, 100, 3, 3], [2 ** 31 - 1, -2 ** 31, 0, 99]],
                                 dtype=torch.int32), 2)
    assert torch.isneginf(lp[0, :2]).all() and lp[0, 2] == lp[0, 3]


def test_many_ids():
    run(make(5, 2, 5000), torch.randint(0, 5000, (2, 3001), dtype=torch.int32), 1)


def test_signed_zeros_are_equal():
    z = torch.zeros(1, 40)
    z[0, ::2] = -0.0
    _, _, top, _ = dsa.token_logprobs(z.to(DEV), top_k=32)
    assert top[0].tolist() == list(range(32))


@pytest.mark.parametrize("V", [64, 20000])
@pytest.mark.parametrize("bad", ["nan", "inf", "none"])
def test_rows_without_a_distribution_are_nan_alone(bad, V):
    z = make(6, 3, V)
    if bad == "none":
        z[1] = -float("inf")
    else:
        z[1, V // 3] = float(bad)
    lp, ent, top, tlp = dsa.token_logprobs(z.to(DEV), torch.zeros(3, 2, dtype=torch.int32,
                                                                  device=DEV), top_k=6)
    for t in (lp, ent, tlp):
        assert torch.isnan(t[1]).all() and torch.isfinite(t[0]).all() and torch.isfinite(t[2]).all()
    assert bool(((top >= 0) & (top < V)).all())


def test_what_is_not_asked_for_is_none():
    z = make(7, 2, 64).to(DEV)
    assert dsa.token_logprobs(z)[0] is None and dsa.token_logprobs(z)[2] is None
    assert dsa.token_logprobs(z, top_k=1, entropy=False)[1] is None


def test_guards_streams_and_graphs():
    z = make(8, 9, 30001)
    zd = z.to(DEV)
    ids = torch.randint(0, 30001, (9, 3), dtype=torch.int32, device=DEV)
    want = dsa.token_logprobs(zd, ids, top_k=7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.token_logprobs(zd, ids, top_k=7, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = dsa.token_logprobs(zd, ids, top_k=7)
    zd.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, dsa.token_logprobs(zd, ids, top_k=7)))
    pinned = dsa.token_logprobs(z.to(DEV), ids.cpu().pin_memory(), top_k=7)
    assert all(torch.equal(a, b) for a, b in zip(pinned, want))
    with pytest.raises(ValueError):
        dsa.token_logprobs(z.pin_memory())


def test_rows_past_32_bits():
    """More than 2^32 bytes of logits: the last row."""
    B, V = 4200, 262144
    z = torch.zeros(B, V, device=DEV)
    z[-1] = make(9, 1, V)[0].to(DEV)
    ids = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    lp, ent, top, tlp = dsa.token_logprobs(z, ids, top_k=3)
    _, rent, rtop, _ = OT.logprobs(z[-1].double().cpu().numpy(), [0], 3)
    assert top[-1].tolist() == list(rtop) and abs(float(ent[-1]) - rent) <= 4e-5 * (1 + rent)
    assert top[-2].tolist() == [0, 1, 2]


def check_shifted(z, ids, K, T, rows):
    """`rows` of z against the oracle, whose rows are less their largest logit. That changes nothing,
    and beside a large one its own ln S would be lost: -3.4e38 + 1.6 is -3.4e38 in 64 bits too."""
    lp, ent, top, tlp = dsa.token_logprobs(z.to(DEV), ids.to(DEV), top_k=K, temperature=T)
    for b in rows:
        row = z[b].double().numpy()
        rlp, rent, rtop, rtlp = OT.logprobs(row - row.max(), ids[b].tolist(), K, T)
        for got, ref in ((lp[b], rlp), (tlp[b] if K else lp[b, :0], rtlp)):
            got = got.double().cpu().numpy()
            far = ref < -3.4e38                # not an fp32 number
            assert np.all(np.isneginf(got[far]) | (got[far] < -3.4e38))
            bound = 4e-5 + 2.0 ** -21 * np.abs(ref)
            assert np.all(np.abs(got[~far] - ref[~far]) <= bound[~far]), (b, K, T)
        assert abs(float(ent[b]) - rent) <= 4e-5 * (1 + rent), (b, K, T)
        if K:
            assert top[b].tolist() == list(rtop), (b, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V", [(4, 5), (4, 1000), (3, 50001), (4, 151936), (200, 45001)])
def test_logits_as_large_as_the_type(B, V, dtype):
    """Rows masked with the type's lowest value, in part and whole, and rows up to its largest:
    z is finite, z log2(e) is not."""
    low = torch.finfo(dtype).min
    z = make(V, B, V, dtype=dtype)
    z[0] = low                                   # all alike: -ln V
    z[1, torch.arange(V) % 7 != 3] = low         # a mask
    z[2] = low
    z[2, V // 2] = -low                          # one certain token, the others 2e38 and more away
    z[2, V // 3] = 0
    if B > 3:
        z[3] = low * 0.75
        z[3, 1::2] = low                         # far apart, both past the range of z log2(e)
    ids = torch.tensor([[0, V - 1, V // 2, 3 % V]] * B, dtype=torch.int32)
    if B > 4:
        z[4:] = z[0]
        z[B - 1] = z[1]
    for K in (0, 1, min(5, V), min(32, V)):
        for T in (1.0, 1.25):
            check_shifted(z, ids, K, T, sorted({0, 1, 2, min(3, B - 1), B - 1}))


@pytest.mark.parametrize("V", [5, 1000, 50001, 151936])
@pytest.mark.parametrize("at", [-1e4, -1e6, 11629080.0, -11629080.0, 1e8, -1e9, 1e10, -1e30, 1e38])
def test_rows_of_large_logits(at, V):
    """All logits near one large value, at any size of it: about 1.16e7 on both sides of 2^24 in base 2."""
    gen = torch.Generator().manual_seed(V)
    step = float(np.spacing(np.float32(abs(at))))
    z = at + step * torch.randint(-3, 4, (4, V), generator=gen).double()
    z[0] = at
    z[1, V // 2] = 0.0                           # and one far from the others
    z[2, : V // 2] = -float("inf")
    ids = torch.tensor([[0, V - 1, V // 2, 3 % V]] * 4, dtype=torch.int32)
    for K in (0, min(5, V)):
        for T in (1.0, 0.8, 3.0):
            if abs(at) / T < 3.4e38:
                check_shifted(z.float(), ids, K, T, range(4))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mask", [-1e4, -1e7, -1e9, -1e10, -1e30, None, -float("inf")])
@pytest.mark.parametrize("B,V", [(3, 40), (3, 20000), (2, 151936), (200, 50001)])
def test_rows_masked_to_a_few_tokens(B, V, mask, dtype):
    """All but a few logits (or one, the last) at a large negative value, some at -inf beside it."""
    z = make(V, B, V, dtype=dtype)
    keep = torch.zeros(V, dtype=torch.bool)
    keep[[0, V // 3, V // 2 + 1, V - 1]] = True
    z[:, ~keep] = torch.finfo(dtype).min if mask is None else mask
    z[1, : V - 1] = z[1, 1]
    z[0, 5: V // 3: 2] = -float("inf")
    ids = torch.tensor([[0, V - 1, V // 2, 1]] * B, dtype=torch.int32)
    for K in (0, 4):
        check_shifted(z, ids, K, 1.0, (0, 1, B - 1))


def gpu_reference(z, ids, T):
    """The definition in float64 torch on the GPU: (log probabilities, entropy, order of the ids)."""
    lp = torch.log_softmax(z.double() / T, 1)
    entropy = -(lp.exp() * lp).sum(1)
    return lp, lp.gather(1, ids.long()), entropy, torch.sort(z.float(), dim=1, descending=True,
                                                           stable=True).indices


def check_rows(z, vocab, K, T):
    """Every row of z (on the GPU), K best of the first `vocab` logits."""
    gen = torch.Generator().manual_seed(K)
    ids = torch.randint(0, vocab, (z.shape[0], 3), generator=gen, dtype=torch.int32).to(DEV)
    lp, ent, top, tlp = dsa.token_logprobs(z, ids, top_k=K, temperature=T, vocab=vocab)
    all_lp, rlp, rent, order = gpu_reference(z[:, :vocab], ids, T)
    for got, ref in ((lp, rlp), (tlp, all_lp.gather(1, order[:, :K]))):
        assert bool(((got.double() - ref).abs() <= 4e-5 + 2.0 ** -21 * ref.abs()).all())
    assert bool(((ent.double() - rent).abs() <= 4e-5 * (1 + rent)).all())
    assert torch.equal(top.long(), order[:, :K])


@pytest.mark.parametrize("K", [1, 8, 9, 32])
@pytest.mark.parametrize("B,V,ld,dtype", [
    (20, 65537, 65537, torch.float32), (60, 65537, 65537, torch.float32),
    (120, 65537, 65539, torch.float32), (60, 131072, 131072, torch.bfloat16),
    (120, 131071, 131073, torch.bfloat16), (152, 262144, 262144, torch.bfloat16)])
def test_every_cluster_of_few_rows(B, V, ld, dtype, K):
    """Rows over clusters of 16, 8 and 4 CTAs."""
    check_rows(make(B + K, B, ld, dtype=dtype).to(DEV), V, K, 0.8)


@pytest.mark.parametrize("K", [1, 8, 9, 32])
@pytest.mark.parametrize("B,V,ld,dtype", [
    (430, 131072, 131072, torch.float32), (430, 131001, 131003, torch.bfloat16),
    (650, 50257, 50304, torch.bfloat16), (700, 40003, 40003, torch.float32),
    (310, 262144, 262144, torch.bfloat16), (900, 7000, 7001, torch.float32)])
def test_large_batches_of_rows(B, V, ld, dtype, K):
    """Several rows to a CTA, one after the other; long ones are read again in several pieces."""
    check_rows(make(B + K, B, ld, dtype=dtype).to(DEV), V, K, 1.3)
