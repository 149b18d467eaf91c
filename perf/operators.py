"""The operators of one verification step of tree-structured speculative decoding, as measured cases.

A draft gives every sequence a tree of N candidate tokens; one pass of the target model scores all of
them. Around the decode step's operators that takes four: rotating the nodes' queries and keys
(``rope``), attention of every node over the cached prefix and its ancestors (``attn``), the log
probabilities that accept or grow drafts (``logprobs``), and moving the accepted path's keys and values
into the cache (``commit``). Each case names its operator in ``op``.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one interactive sequence, a short context and a small tree: launch latency counts
        dict(name="attn_chat_512", op="attn", B=1, Hq=16, Hkv=8, D=128, N=8, lens="fixed", a=512, b=512,
             softcap=0.0, alibi=False, window=0, ragged=False),
        # one sequence over a 131072-token context, a tree of 26 nodes: the cache's bandwidth
        dict(name="attn_long_131k", op="attn", B=1, Hq=32, Hkv=8, D=128, N=26, lens="fixed", a=131072,
             b=131072, softcap=0.0, alibi=False, window=0, ragged=False),
        # a ragged batch, scores capped by a tanh, trees of up to 16 nodes
        dict(name="attn_batch_cap", op="attn", B=32, Hq=32, Hkv=8, D=128, N=16, lens="uniform", a=512, b=8192,
             softcap=50.0, alibi=False, window=0, ragged=True),
        # a serving mix of many short contexts, one new token each, a bias that falls with distance, head_dim 64
        dict(name="attn_single_alibi_d64", op="attn", B=192, Hq=16, Hkv=4, D=64, N=1, lens="geometric", a=2048,
             b=32768, softcap=0.0, alibi=True, window=0, ragged=False),
        # full trees of 64 nodes on groups of eight query heads, a sliding window of 4095: the tensor cores
        dict(name="attn_wide_window", op="attn", B=16, Hq=64, Hkv=8, D=128, N=64, lens="uniform", a=1000, b=9000,
             softcap=0.0, alibi=False, window=4095, ragged=False),
        # the rotation of one sequence's tree
        dict(name="rope_chat", op="rope", B=1, Hq=16, Hkv=8, D=128, N=8, layout="neox", norm=True, theta=1e6,
             far=512, ragged=False),
        # the rotation of a batch of full trees
        dict(name="rope_batch", op="rope", B=96, Hq=32, Hkv=8, D=128, N=64, layout="interleaved", norm=True,
             theta=5e5, far=131072, ragged=True),
        # the next token's alternatives for one row of a large vocabulary
        dict(name="logprobs_row", op="logprobs", rows=1, V=151936, ld=151936, C=1, K=20, bf16=False, temp=1.0),
        # every node of a batch of trees: each node's children's log probabilities and the best alternatives
        dict(name="logprobs_trees", op="logprobs", rows=512, V=131072, ld=131072, C=4, K=8, bf16=False, temp=0.7),
        # scoring a text: bf16 logits of an odd vocabulary in rows padded to the projection's multiple of 128
        dict(name="logprobs_text_bf16", op="logprobs", rows=2047, V=50257, ld=50304, C=1, K=1, bf16=True, temp=1.0),
        # the accepted path of a batch of trees into the cache
        dict(name="commit_batch", op="commit", B=32, Hkv=8, D=128, N=16, T=8192),
        # a large batch of full trees
        dict(name="commit_wide", op="commit", B=256, Hkv=4, D=128, N=64, T=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rope", "logprobs", "logprobs", "commit"])
    if op == "attn":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
        N, D = _log_int(rng, 1, 64), rng.choice([64, 128])
        top = _log_int(rng, 16, 131072)
        # at most about 2^20 cached rows of all heads together, and the largest listed case's arithmetic
        B = max(1, min(_log_int(rng, 1, 192), (1 << 20) // (Hkv * top), (1 << 29) // (Hkv * G * N * top)))
        kind = rng.choice(["fixed", "uniform", "geometric"])
        a = top if kind == "fixed" else max(1, top // rng.choice([4, 16]))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, N=N, lens=kind, a=a, b=top,
                    softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.3,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, top)]), ragged=rng.random() < 0.5)
    if op == "rope":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
        return dict(op=op, B=_log_int(rng, 1, 64), Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]),
                    N=_log_int(rng, 1, 64), layout=rng.choice(["neox", "interleaved"]),
                    norm=rng.random() < 0.5, theta=rng.choice([1e4, 5e5, 1e6]), far=_log_int(rng, 1, 131072),
                    ragged=rng.random() < 0.5)
    if op == "logprobs":
        V = _log_int(rng, 1000, 262144)
        ld = rng.choice([V, (V + 127) // 128 * 128])
        rows = max(1, min(_log_int(rng, 1, 2048), (1 << 26) // V))
        return dict(op=op, rows=rows, V=V, ld=ld, C=rng.choice([1, 2, 5, 16]), K=rng.choice([0, 1, 5, 20, 32]),
                    bf16=rng.random() < 0.5, temp=rng.choice([1.0, 1.0, 0.7, 1.3]))
    N = _log_int(rng, 2, 64)
    return dict(op=op, B=_log_int(rng, 1, 128), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), N=N,
                T=_log_int(rng, 2 * N, 2048))


# ----------------------------------------------------------------- inputs ---
def _lengths(case):
    """The lengths of a case's sequences, in increasing order: the same for every seed (they are shuffled
    by the seed), so that a case's work is fixed."""
    B, a, b = case["B"], case["a"], case["b"]
    u = (np.arange(B) + 0.5) / B
    if case["lens"] == "fixed":
        x = np.full(B, a)
    elif case["lens"] == "uniform":
        x = a + (b - a) * u
    else:
        x = np.minimum(-a * np.log1p(-u), b)
    return np.maximum(1, np.floor(x)).astype(np.int64)


def _node_counts(case):
    """Nodes per sequence: all N, or (ragged) between half of N and N; shuffled by the seed."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return np.full(B, N, dtype=np.int64)
    return np.maximum(1, np.ceil(N * (0.5 + 0.5 * (np.arange(B) + 0.5) / B))).astype(np.int64)


def _trees(rng, B, N):
    """Random trees: node 0 is the root, node n's parent one of the four nodes before it. Ancestor
    masks (bit j of word n: node n sees node j, itself included) and depths."""
    mask = np.zeros((B, N), dtype=np.uint64)
    depth = np.zeros((B, N), dtype=np.int64)
    row = np.arange(B)
    mask[:, 0] = 1
    for n in range(1, N):
        parent = rng.integers(max(0, n - 4), n, size=B)
        mask[:, n] = mask[row, parent] | np.uint64(1 << n)
        depth[:, n] = depth[row, parent] + 1
    return mask.view(np.int64), depth


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "attn":
        B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
        lens = rng.permutation(_lengths(case))
        T = int(lens.max())
        mask, depth = _trees(rng, B, N)
        s["max_len"] = T
        s["lens"], s["n_nodes"] = _i32(lens), _i32(rng.permutation(_node_counts(case)))
        s["mask"] = torch.from_numpy(mask).to(DEV)
        s["pos"] = _i32(lens[:, None] + depth)
        s["q"] = _normal(gen, B, N, Hq, D)
        s["k_cache"], s["v_cache"] = _normal(gen, B, Hkv, T, D), _normal(gen, B, Hkv, T, D)
        s["k_tree"], s["v_tree"] = _normal(gen, B, Hkv, N, D), _normal(gen, B, Hkv, N, D)
        # a slope for every query head, 2^(-8 (h + 1) / Hq)
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32) / Hq)
        s["out"] = torch.zeros(B, N, Hq, D, device=DEV, dtype=torch.bfloat16)
        if own:
            import decode_step_attention_gb300 as dsa
            s["workspace"] = dsa.alloc_tree_workspace(B, N, Hq, Hkv, D, T)
    elif op == "rope":
        B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
        s["q"], s["k_new"], s["v_new"] = (_normal(gen, B, N, h, D) for h in (Hq, Hkv, Hkv))
        w = (1 + 0.1 * _normal(gen, 2, D).float()).bfloat16()
        s["q_norm_w"], s["k_norm_w"] = (w[0].contiguous(), w[1].contiguous()) if case["norm"] else (None, None)
        start = rng.integers(max(0, case["far"] // 2), case["far"] + 1, size=B)
        s["pos"] = _i32(start[:, None] + _trees(rng, B, N)[1])
        s["n_nodes"] = _i32(rng.permutation(_node_counts(case)))
        s["q_out"] = torch.zeros_like(s["q"])
        s["k_tree"] = torch.zeros(B, Hkv, N, D, device=DEV, dtype=torch.bfloat16)
        s["v_tree"] = torch.zeros_like(s["k_tree"])
    elif op == "logprobs":
        rows, V, ld = case["rows"], case["V"], case["ld"]
        # a bell of logits with some hundred favoured tokens per row, as a trained model gives
        z = torch.randn(rows, ld, generator=gen, device=DEV, dtype=torch.float32) * 2.0
        at = torch.randint(0, V, (rows, 128), generator=gen, device=DEV)
        z.scatter_add_(1, at, 6.0 + 3.0 * torch.randn(rows, 128, generator=gen, device=DEV))
        s["logits"] = z.bfloat16() if case["bf16"] else z
        ids = torch.randint(0, V, (rows, case["C"]), generator=gen, device=DEV)
        ids[:, 0] = at[:, 0]
        s["tokens"] = ids.int()
    else:
        B, Hkv, D, N, T = (case[k] for k in ("B", "Hkv", "D", "N", "T"))
        s["k_cache"], s["v_cache"] = _normal(gen, B, Hkv, T, D), _normal(gen, B, Hkv, T, D)
        s["k_tree"], s["v_tree"] = _normal(gen, B, Hkv, N, D), _normal(gen, B, Hkv, N, D)
        s["lens"] = _i32(rng.integers(0, T - N + 1, size=B))
        # an increasing path of nodes of every accepted length, one at least
        path = np.sort(rng.random((B, N)).argsort(axis=1), axis=1)
        count = rng.permutation(_path_counts(case))
        keep = rng.random((B, N)).argsort(axis=1)
        for b in range(B):
            path[b, :count[b]] = np.sort(keep[b, :count[b]])
        s["path"], s["n_path"] = _i32(path), _i32(count)
    return s


def _path_counts(case):
    return 1 + np.arange(case["B"]) % case["N"]


# -------------------------------------------------------------------- run ---
def run(s):
    op = s["op"]
    if own:
        import decode_step_attention_gb300 as dsa
        if op == "attn":
            return dsa.gqa_tree_attn(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["k_tree"], s["v_tree"],
                                     s["mask"], n_nodes=s["n_nodes"], pos=s["pos"], max_len=s["max_len"],
                                     workspace=s["workspace"], out=s["out"], softcap=s["softcap"],
                                     slopes=s["slopes"] if s["alibi"] else None, window=s["window"])
        if op == "rope":
            dsa.qknorm_rope_tree(s["q"], s["k_new"], s["v_new"], s["k_tree"], s["v_tree"], s["pos"], s["theta"],
                                 layout=s["layout"], q_norm_w=s["q_norm_w"], k_norm_w=s["k_norm_w"],
                                 n_nodes=s["n_nodes"], q_out=s["q_out"])
            return s["q_out"], s["k_tree"], s["v_tree"]
        if op == "logprobs":
            lp, ent, ids, top = dsa.token_logprobs(s["logits"], s["tokens"], top_k=s["K"], temperature=s["temp"],
                                                   vocab=s["V"])
            return (lp, ent, ids, top) if s["K"] else (lp, ent)
        dsa.tree_commit(s["k_tree"], s["v_tree"], s["path"], s["n_path"], s["k_cache"], s["v_cache"], s["lens"])
        return s["k_cache"], s["v_cache"]
    return {"attn": _attn, "rope": _rope, "logprobs": _logprobs, "commit": _commit}[op](s)


def _attn(s):
    B, N, Hq, D = s["q"].shape
    Hkv, T = s["k_cache"].shape[1:3]
    G = Hq // Hkv
    f32 = torch.float32
    keys = torch.cat([s["k_cache"], s["k_tree"]], 2).to(f32)
    vals = torch.cat([s["v_cache"], s["v_tree"]], 2).to(f32)
    # query rows of a KV head: (head in its group, node)
    q = s["q"].to(f32).view(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, D)
    z = (q @ keys.transpose(2, 3)).view(B, Hkv, G, N, T + N) * (1.0 / math.sqrt(D))
    if s["softcap"]:
        z = torch.tanh(z / s["softcap"]) * s["softcap"]
    slot = torch.arange(T, device=DEV)
    node = torch.arange(N, device=DEV)
    pos = s["pos"].long()
    far = pos[:, :, None] - torch.cat([slot.expand(B, T), pos], 1)[:, None, :]  # [B, N, T + N]
    if s["alibi"]:
        z = z - s["slopes"].view(1, Hkv, G, 1, 1) * far[:, None, None].to(f32)
    real = node < s["n_nodes"][:, None]                                         # [B, N]
    in_cache = (slot < s["lens"][:, None])[:, None, :].expand(B, N, T)
    in_tree = ((s["mask"][:, :, None] >> node) & 1).bool() & real[:, None, :]
    seen = torch.cat([in_cache, in_tree], 2)
    if s["window"]:
        seen = seen & (far < s["window"])
    z = torch.where(seen[:, None, None], z, torch.full((), -math.inf, device=DEV))
    e = torch.exp(z - z.amax(-1, keepdim=True))
    o = (e.view(B, Hkv, G * N, T + N) @ vals).view(B, Hkv, G, N, D) / e.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    return torch.where(real[:, :, None, None], o, torch.zeros((), device=DEV)).bfloat16()


def _turn(x, w, cos, sin, layout, eps=1e-6):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    if layout == "neox":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _rope(s):
    B, N, Hq, D = s["q"].shape
    freq = s["theta"] ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    angle = s["pos"].double()[:, :, None, None] * freq                          # far positions: in 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    real = (torch.arange(N, device=DEV) < s["n_nodes"][:, None])
    q = _turn(s["q"], s["q_norm_w"], cos, sin, s["layout"]).bfloat16()
    k = _turn(s["k_new"], s["k_norm_w"], cos, sin, s["layout"]).bfloat16().transpose(1, 2)
    rows, cols = real[:, :, None, None], real[:, None, :, None]
    return (torch.where(rows, q, s["q_out"]), torch.where(cols, k, s["k_tree"]),
            torch.where(cols, s["v_new"].transpose(1, 2), s["v_tree"]))


def _logprobs(s):
    V = s["V"]
    raw = s["logits"][:, :V].float()
    z = raw / s["temp"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + total.log()
    lp = z.gather(1, s["tokens"].long()) - lse
    entropy = total.log()[:, 0] - (e * (z - top)).sum(1) / total[:, 0]
    if not s["K"]:
        return lp, entropy
    # the best K: a key that orders by value, then by the lower id
    bits = raw.view(torch.int32).long()
    bits = torch.where(bits < 0, bits ^ 0x7fffffff, bits)
    key = (bits << 18) + (262143 - torch.arange(V, device=DEV))
    ids = 262143 - (key.topk(s["K"], dim=1).values & 262143)
    return lp, entropy, ids.int(), z.gather(1, ids) - lse


def _commit(s):
    B, N = s["path"].shape
    i = torch.arange(N, device=DEV)
    row = torch.arange(B, device=DEV)[:, None]
    slot = s["lens"].long()[:, None] + i
    live = (i < s["n_path"][:, None])[:, :, None, None]
    path = s["path"].long()
    for cache, tree in ((s["k_cache"], s["k_tree"]), (s["v_cache"], s["v_tree"])):
        cache[row, :, slot] = torch.where(live, tree[row, :, path], cache[row, :, slot])
    return s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------- work ---
def work(case):
    op = case["op"]
    if op == "attn":
        lens, nodes = _lengths(case), _node_counts(case)
        if case["window"]:
            lens = np.minimum(lens, max(0, case["window"] - 1))
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        # sorted against sorted: the seed pairs lengths and node counts at random
        pairs = float(lens.sum()) * float(nodes.mean()) + float((nodes * (nodes + 1) / 2).sum())
        kv = 4.0 * Hkv * D * (float(lens.sum()) + float(nodes.sum()))
        return {"bytes": kv + 4.0 * Hq * D * float(nodes.sum()), "flops": 4.0 * Hq * D * pairs}
    if op == "rope":
        n = float(_node_counts(case).sum())
        elems = n * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
        return {"bytes": 4.0 * elems, "flops": 8.0 * elems}
    if op == "logprobs":
        n = case["rows"] * case["V"]
        return {"bytes": n * (2.0 if case["bf16"] else 4.0) + case["rows"] * (8.0 * case["C"] + 4 + 8.0 * case["K"]),
                "flops": 6.0 * n}
    rows = float(_path_counts(case).sum()) * case["Hkv"]
    return {"bytes": 2 * 4.0 * rows * case["D"], "flops": 0.0}


# ------------------------------------------------------------------ exact ---
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn":
        B, N, Hq, D = s["q"].shape
        G = Hq // s["Hkv"]
        out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=DEV)
        for b in range(B):
            L, n = int(s["lens"][b]), int(s["n_nodes"][b])
            K = torch.cat([s["k_cache"][b, :, :L], s["k_tree"][b, :, :n]], 1).double()
            V = torch.cat([s["v_cache"][b, :, :L], s["v_tree"][b, :, :n]], 1).double()
            words = s["mask"][b].tolist()
            allow = torch.zeros(n, L + n, dtype=torch.bool)
            allow[:, :L] = True
            for i in range(n):
                for j in range(n):
                    allow[i, L + j] = bool((words[i] >> j) & 1)
            kpos = torch.cat([torch.arange(L), s["pos"][b, :n].cpu().long()])
            dist = s["pos"][b, :n].cpu().long()[:, None] - kpos[None]
            if case["window"]:
                allow &= dist < case["window"]
            allow, dist = allow.to(DEV), dist.to(DEV).double()
            for h in range(Hq):
                x = s["q"][b, :n, h].double() @ K[h // G].T / math.sqrt(D)
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if case["alibi"]:
                    x = x - s["slopes"][h].double() * dist
                x = x.masked_fill(~allow, -math.inf)
                out[b, :n, h] = torch.softmax(x, -1) @ V[h // G]
        return out
    if op == "rope":
        B, N, Hq, D = s["q"].shape
        i = np.arange(D // 2)
        f = np.power(float(case["theta"]), -2.0 * i / D)
        phi = s["pos"].cpu().numpy().astype(np.float64)[..., None] * f
        turn = torch.complex(torch.from_numpy(np.cos(phi)), torch.from_numpy(np.sin(phi)))[:, :, None]

        def rotated(x, w):
            x = x.cpu().double()
            if w is not None:
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.cpu().double()
            if case["layout"] == "neox":
                c = torch.complex(x[..., :D // 2], x[..., D // 2:]) * turn
                return torch.cat([c.real, c.imag], -1)
            c = torch.view_as_complex(x.unflatten(-1, (D // 2, 2)).contiguous()) * turn
            return torch.view_as_real(c).flatten(-2)

        q, k = rotated(s["q"], s["q_norm_w"]), rotated(s["k_new"], s["k_norm_w"]).transpose(1, 2).clone()
        v = s["v_new"].cpu().double().transpose(1, 2).clone()
        for b in range(B):
            n = int(s["n_nodes"][b])
            q[b, n:], k[b, :, n:], v[b, :, n:] = 0, 0, 0
        return q, k, v
    if op == "logprobs":
        z = s["logits"][:, :case["V"]].double() / case["temp"]
        lp = torch.log_softmax(z, 1)
        p = lp.exp()
        given = lp.gather(1, s["tokens"].long())
        entropy = -(p * lp).sum(1)
        if not case["K"]:
            return given, entropy
        order = torch.sort(s["logits"][:, :case["V"]].float(), dim=1, descending=True, stable=True).indices
        ids = order[:, :case["K"]]
        return given, entropy, ids.int(), lp.gather(1, ids)
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    for b, (at, n) in enumerate(zip(s["lens"].tolist(), s["n_path"].tolist())):
        nodes = s["path"][b, :n].long()
        k[b, :, at:at + n] = s["k_tree"][b][:, nodes]
        v[b, :, at:at + n] = s["v_tree"][b][:, nodes]
    return k, v
