"""Cases that measure the front of an attention layer (rotary positions, per-head
norms of queries and keys) and attention for a tree of drafted tokens.

``run`` computes a case in its plain form (elementary torch operations in 32 bits,
angles in 64) or, with ``own`` set, by the calls a user of the package makes.

Sizes: 16 query heads over 2 key heads of 128 dims with an indexer of 4 heads of
64, and 4 heads over 1 of 64 dims, are the layer's deployed and tiny
configurations; lengths run from one token to 128K, odd ones among them.
"""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-6
#: dims a frequency pair turns by at position p: p * base^(-2i/rot), stretched
#: by parts for contexts longer than the trained length
BASE, FACTOR, TRAINED, FAST, SLOW = 1.0e6, 8.0, 32768, 32.0, 1.0


# ------------------------------------------------------------------- cases --

def listed():
    """The cases: each a real step of the layer."""
    return [
        # one decode step of 64 sequences: the indexer's queries, half of each head turned
        dict(name="rope-index-step", op="rope", B=64, T=1, H=4, D=64, rot=32, layout="half",
             scaling="by-parts", dtype="bf16", transpose=False, far=1000000),
        # gradients of rotated queries in fp32, as the sparse backward leaves them; odd length
        dict(name="rope-grad-32", op="rope", B=2, T=4099, H=16, D=128, rot=64,
             layout="interleaved", scaling="none", dtype="fp32", transpose=True, far=0),
        # one decode step of 64 sequences: packed projection to queries and caches
        dict(name="norm-rope-step", op="norm_rope", B=64, T=1, Hq=16, Hkv=2, D=128, rot=128,
             layout="half", scaling="by-parts", L=2048),
        # a 32K prompt's projection to queries and caches
        dict(name="norm-rope-prompt", op="norm_rope", B=1, T=32768, Hq=16, Hkv=2, D=128, rot=128,
             layout="half", scaling="none", L=33000),
        # training on short sequences, tiny configuration, 16-bit gradients
        dict(name="norm-rope-grad-tiny", op="norm_rope_grad", B=2, T=1001, Hq=4, Hkv=1, D=64,
             rot=32, layout="interleaved", scaling="none", dtype="bf16"),
        # training on a 32K sequence, fp32 gradients from the sparse backward
        dict(name="norm-rope-grad-32k", op="norm_rope_grad", B=1, T=32768, Hq=16, Hkv=2, D=128,
             rot=128, layout="half", scaling="by-parts", dtype="fp32"),
        # a short chat, a few drafts: latency
        dict(name="tree-short", op="dense_tree", B=1, N=7, Hq=4, Hkv=1, D=64, prefix=1003,
             ragged=False),
        # a serving batch of unequal contexts
        dict(name="tree-batch", op="dense_tree", B=32, N=8, Hq=16, Hkv=2, D=128, prefix=16384,
             ragged=True),
        # one long document, a small tree
        dict(name="tree-long", op="dense_tree", B=1, N=16, Hq=16, Hkv=2, D=128, prefix=131072,
             ragged=False),
        # wide trees: the matrix products weigh more than the cache's bytes
        dict(name="tree-wide", op="dense_tree", B=4, N=64, Hq=16, Hkv=2, D=128, prefix=65536,
             ragged=False),
        # drafts that read their selected blocks only, tiny configuration
        dict(name="sparse-tree-tiny", op="sparse_tree", B=2, N=5, Hq=4, Hkv=1, D=64, prefix=4093,
             budget=512, ragged=True),
        # the deployed budget over long caches
        dict(name="sparse-tree-64k", op="sparse_tree", B=8, N=16, Hq=16, Hkv=2, D=128,
             prefix=65539, budget=2048, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["rope", "norm_rope", "norm_rope_grad", "dense_tree", "dense_tree",
                     "sparse_tree"])
    lay = rng.choice(["half", "interleaved"])
    sca = rng.choice(["none", "linear", "by-parts"])
    Hkv = rng.choice([1, 2, 4])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    if op == "rope":
        D = rng.choice([32, 64, 128])
        H = rng.choice([1, 2, 4, 16])
        tokens = _log(rng, 1, 4000000 // (H * D) * 4)
        B = rng.choice([1, 2, 3, 8])
        return dict(op=op, B=B, T=max(1, tokens // B), H=H, D=D, rot=rng.choice([D // 4, D // 2, D]),
                    layout=lay, scaling=sca, dtype=rng.choice(["bf16", "fp32"]),
                    transpose=rng.random() < 0.5, far=rng.choice([0, 1000, 1000000]))
    if op in ("norm_rope", "norm_rope_grad"):
        tokens = _log(rng, 1, 64000000 // ((Hq + 2 * Hkv) * D))
        B = rng.choice([1, 2, 3, 16])
        T = max(1, min(tokens // B, 32768))
        c = dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D // 4, D // 2, D]),
                 layout=lay, scaling=sca)
        if op == "norm_rope":
            c["L"] = T + rng.randint(0, 300)
        else:
            c["dtype"] = rng.choice(["bf16", "fp32"])
        return c
    N = _log(rng, 1, 64)
    B = _log(rng, 1, 32)
    if op == "dense_tree":
        most = min(131072, 2 ** 31 // (N * Hq * B), 2 ** 28 // (B * Hkv * D))
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D,
                    prefix=_log(rng, 1, max(2, most)) - 1, ragged=rng.random() < 0.5)
    B = min(B, max(1, 128 // N))
    most = min(65536, 2 ** 27 // (B * Hkv * D))
    return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, prefix=_log(rng, 1, max(2, most)),
                budget=rng.choice([64, 512, 2048]), ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs --

def _freq(rot, scaling):
    """Radians per position of each pair, and the factor on rotated dims."""
    f = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return [x / FACTOR for x in f], 1.0
    turn = lambda beta: rot * math.log(TRAINED / (beta * 2 * math.pi)) / (2 * math.log(BASE))
    lo, hi = max(math.floor(turn(FAST)), 0), min(math.ceil(turn(SLOW)), rot - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rot // 2)]
    return [x / FACTOR * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(FACTOR) + 1.0


def _lens(c):
    """Committed tokens and drafts of each sequence."""
    B, P, N = c["B"], c["prefix"], c["N"]
    if not c["ragged"]:
        return [P] * B, [N] * B
    return ([P - (P * b) // (2 * B) for b in range(B)],
            [max(1, N - (3 * b) % max(1, N // 2 + 1)) for b in range(B)])


def _windows(blocks, keep, N):
    """A tree's rows keep a common half and each a run of the other blocks, in a
    shuffled order: (common, first and length of each row's run)."""
    if blocks <= keep:
        return blocks, [(0, 0)] * N
    common = keep // 2
    rest, run_ = blocks - common, keep - common
    return common, [((i * rest) // N, run_) for i in range(N)]


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {}
    if c["op"] in ("rope", "norm_rope", "norm_rope_grad"):
        f, s["mscale"] = _freq(c["rot"], c["scaling"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    B = c["B"]
    if c["op"] == "rope":
        s["x"] = _randn(g, B, c["T"], c["H"], c["D"],
                        dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=DEV)
        s["pos"] = first + torch.arange(c["T"], device=DEV)
    elif c["op"] == "norm_rope":
        T, Hq, Hkv, D, L = c["T"], c["Hq"], c["Hkv"], c["D"], c["L"]
        packed = _randn(g, B, T, (Hq + 2 * Hkv) * D)
        s["q"] = packed[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = packed[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        s["v"] = packed[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
        s["q_weight"] = 1 + 0.1 * _randn(g, D, dtype=torch.float32)
        s["k_weight"] = 1 + 0.1 * _randn(g, D, dtype=torch.float32)
        s["k_cache"], s["v_cache"] = _randn(g, B, L, Hkv, D), _randn(g, B, L, Hkv, D)
        first = torch.randint(0, L - T + 1, (B, 1), generator=g, device=DEV)
        s["pos"] = first + torch.arange(T, device=DEV)
        s["slot"] = s["pos"].clone()
    elif c["op"] == "norm_rope_grad":
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        t = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["q"], s["k"] = _randn(g, B, T, Hq, D), _randn(g, B, T, Hkv, D)
        s["d_q"], s["d_k"] = _randn(g, B, T, Hq, D, dtype=t), _randn(g, B, T, Hkv, D, dtype=t)
        s["q_weight"] = 1 + 0.1 * _randn(g, D, dtype=torch.float32)
        s["k_weight"] = 1 + 0.1 * _randn(g, D, dtype=torch.float32)
        s["pos"] = torch.arange(T, device=DEV).expand(B, T).contiguous()
    else:
        N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
        s["prefix"], s["drafts"] = _lens(c)
        L = c["prefix"] + N
        s["q"] = 2 * _randn(g, B, N, Hq, D)
        s["k_cache"], s["v_cache"] = _randn(g, B, L, Hkv, D), _randn(g, B, L, Hkv, D)
        s["seqlens"] = torch.tensor([p + n for p, n in zip(s["prefix"], s["drafts"])],
                                    dtype=torch.int32, device=DEV)
        s["n_draft"] = torch.tensor(s["drafts"], dtype=torch.int32, device=DEV)
        # drafts grow mostly by chains: a parent a little before its child
        i = torch.arange(N, device=DEV)
        back = (torch.rand(B, N, generator=g, device=DEV) ** 3 * (i + 1)).long()
        s["parent"] = (i - 1 - back).clamp_min(-1).int()
        if c["op"] == "sparse_tree":
            keep = c["budget"] // 4 - 1
            s["sel"] = torch.full((B, N, keep + 1), -1, dtype=torch.int32, device=DEV)
            for b in range(B):
                blocks = s["prefix"][b] // 4
                order = torch.randperm(blocks, generator=g, device=DEV).int()
                common, runs = _windows(blocks, keep, N)
                for n, (first, length) in enumerate(runs):
                    own_ = common + (first + torch.arange(length, device=DEV)) % max(1, blocks - common)
                    row = torch.cat([order[:common], order[own_]]).sort().values
                    s["sel"][b, n, :row.numel()] = row
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import block_sparse_long_10_b200 as qsa
        s["qsa"] = qsa
        c, op, B = case, case["op"], case["B"]
        if op == "rope":
            s["y"] = torch.empty_like(s["x"])
        elif op == "norm_rope":
            s["q_out"] = torch.empty(B, c["T"], c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
        elif op == "norm_rope_grad":
            s["dq"], s["dk"] = torch.empty_like(s["d_q"]), torch.empty_like(s["d_k"])
            s["dqw"], s["dkw"] = (torch.empty(c["D"], device=DEV) for _ in range(2))
            s["ws"] = qsa.workspace(qsa.qsa_qk_norm_rope_backward_workspace_size(
                B, c["T"], c["Hq"], c["Hkv"], c["D"]), DEV)
        else:
            s["o"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(B, c["N"], c["Hq"], device=DEV)
            if op == "dense_tree":
                n = qsa.qsa_dense_tree_decode_workspace_size(B, c["N"], c["Hq"], c["Hkv"], c["D"])
            else:
                n = qsa.qsa_sparse_tree_decode_workspace_size(B, c["N"], c["Hq"], c["D"], 4,
                                                              c["budget"])
            s["ws"] = qsa.workspace(n, DEV)
    return s


# -------------------------------------------------------------- plain forms --

def _turn(x, pos, freq, layout, mscale, transpose):
    """x [B,T,H,D] fp32 with its first 2 * len(freq) dims turned by pos * freq."""
    rot = 2 * freq.numel()
    angle = pos.double()[..., None] * freq
    cos = (angle.cos() * mscale).float()[:, :, None]
    sin = (angle.sin() * mscale).float()[:, :, None]
    if transpose:
        sin = -sin
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _norm(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _norm_grad(dy, x, weight, pos, freq, layout, mscale):
    dz = _turn(dy.float(), pos, freq, layout, mscale, True)
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dw = (dz * xh).sum((0, 1, 2))
    u = dz * weight
    return (r * (u - xh * (u * xh).mean(-1, keepdim=True))).to(dy.dtype), dw


def _ancestors(parent):
    """[N, N] truth: column j is row i's ancestor or itself."""
    N = parent.numel()
    one = torch.eye(N, device=DEV)
    step = torch.zeros(N, N + 1, device=DEV)
    step[torch.arange(N, device=DEV), parent.long()] = 1  # -1 lands in the last column
    reach = one + step[:, :N]
    for _ in range(max(1, (N - 1).bit_length())):
        reach = (reach @ reach > 0).float()
    return reach > 0


def _attend(q, k, v, ok, scale):
    """q [n,Hq,D], k/v [S,Hkv,D] (or [n,S,Hkv,D]), ok [n,S] -> o [n,Hq,D], lse [n,Hq], fp32."""
    n, Hq, D = q.shape
    Hkv = k.shape[-2]
    q = q.float().unflatten(1, (Hkv, Hq // Hkv))                       # n g h d
    if k.dim() == 3:
        rows = q.permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        x = (rows @ k.permute(1, 2, 0)).unflatten(1, (n, Hq // Hkv)).transpose(0, 1)
    else:
        x = q @ k.permute(0, 2, 3, 1)                                  # n g h S
    x = (x * scale).masked_fill(~ok[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    if v.dim() == 3:
        rows = p.transpose(0, 1).reshape(Hkv, -1, p.shape[-1])
        o = (rows @ v.transpose(0, 1)).unflatten(1, (n, Hq // Hkv)).transpose(0, 1)
    else:
        o = p @ v.transpose(1, 2)
    return o.reshape(n, Hq, D), (top + torch.log(total)).reshape(n, Hq)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "rope":
        return {"y": _turn(s["x"].float(), s["pos"], s["freq"], c["layout"], s["mscale"],
                           c["transpose"]).to(s["x"].dtype)}
    if op == "norm_rope":
        how = (s["pos"], s["freq"], c["layout"], s["mscale"], False)
        b = torch.arange(c["B"], device=DEV)[:, None]
        s["k_cache"][b, s["slot"]] = _turn(_norm(s["k"], s["k_weight"]), *how).bfloat16()
        s["v_cache"][b, s["slot"]] = s["v"]
        return {"q": _turn(_norm(s["q"], s["q_weight"]), *how).bfloat16(),
                "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "norm_rope_grad":
        how = (s["pos"], s["freq"], c["layout"], s["mscale"])
        dq, dqw = _norm_grad(s["d_q"], s["q"], s["q_weight"], *how)
        dk, dkw = _norm_grad(s["d_k"], s["k"], s["k_weight"], *how)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    o = torch.zeros_like(s["q"])
    lse = torch.zeros(s["q"].shape[:3], device=DEV)
    for b, (P, n) in enumerate(zip(s["prefix"], s["drafts"])):
        k, v = s["k_cache"][b, :P + n].float(), s["v_cache"][b, :P + n].float()
        tree = _ancestors(s["parent"][b, :n])
        if op == "dense_tree":
            ok = torch.cat([torch.ones(n, P, dtype=torch.bool, device=DEV), tree], 1)
        else:
            blk = s["sel"][b, :n].long()
            whole = P // 4
            four = torch.arange(4, device=DEV)
            tok = (blk.clamp_min(0)[..., None] * 4 + four).flatten(1)
            live = ((blk >= 0) & (blk < whole))[..., None].expand(-1, -1, 4).flatten(1)
            last = torch.arange(whole * 4, P + n, device=DEV).expand(n, -1)
            tail = torch.ones(n, P - whole * 4, dtype=torch.bool, device=DEV)
            tok, ok = torch.cat([tok, last], 1), torch.cat([live, tail, tree], 1)
            k, v = k[tok], v[tok]
        y, z = _attend(s["q"][b, :n], k, v, ok, c["D"] ** -0.5)
        o[b, :n], lse[b, :n] = y.bfloat16(), z
    return {"o": o, "lse": lse}


# --------------------------------------------------------------------- run --

def run(s):
    """One pass: the plain form, or the package's calls."""
    if not own:
        return _plain(s)
    c, qsa = s["case"], s["qsa"]
    op = c["op"]
    if op == "rope":
        qsa.qsa_rope(s["x"], s["y"], s["freq"], pos=s["pos"], layout=c["layout"],
                     mscale=s["mscale"], transpose=c["transpose"])
        return {"y": s["y"]}
    if op == "norm_rope":
        qsa.qsa_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_cache"], s["freq"], v=s["v"],
                             v_out=s["v_cache"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                             eps=EPS, pos=s["pos"], layout=c["layout"], mscale=s["mscale"],
                             slot=s["slot"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "norm_rope_grad":
        qsa.qsa_qk_norm_rope_backward(s["d_q"], s["d_k"], s["q"], s["k"], s["dq"], s["dk"],
                                      s["freq"], s["ws"], q_weight=s["q_weight"],
                                      k_weight=s["k_weight"], dq_weight=s["dqw"],
                                      dk_weight=s["dkw"], eps=EPS, pos=s["pos"],
                                      layout=c["layout"], mscale=s["mscale"])
        return {"dq": s["dq"], "dk": s["dk"], "dq_weight": s["dqw"], "dk_weight": s["dkw"]}
    if op == "dense_tree":
        qsa.qsa_dense_tree_decode(s["q"], s["k_cache"], s["v_cache"], s["seqlens"], s["parent"],
                                  s["o"], s["ws"], n_draft=s["n_draft"], lse=s["lse"])
    else:
        qsa.qsa_sparse_tree_decode(s["q"], s["k_cache"], s["v_cache"], s["seqlens"], s["sel"],
                                   s["parent"], s["o"], s["ws"], n_draft=s["n_draft"], r=4,
                                   budget=c["budget"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


# -------------------------------------------------------------------- work --

def _union(runs, rest):
    """Blocks of `rest` that the cyclic runs cover together."""
    seen = 0
    reach = 0
    for first, length in sorted(runs):
        seen += max(0, first + length - max(first, reach))
        reach = max(reach, first + length)
    return min(rest, seen)


def work(case):
    """Bytes of each input and output once, and operations."""
    c = case
    op, B, D = c["op"], c["B"], c["D"]
    if op == "rope":
        n = B * c["T"] * c["H"] * D
        return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 8 * B * c["T"],
                "flops": 3 * n}
    if op == "norm_rope":
        n = B * c["T"] * (c["Hq"] + 2 * c["Hkv"]) * D
        return {"bytes": 4 * n + 16 * B * c["T"], "flops": 8 * n}
    if op == "norm_rope_grad":
        n = B * c["T"] * (c["Hq"] + c["Hkv"]) * D
        return {"bytes": n * (2 + 2 * (2 if c["dtype"] == "bf16" else 4)) + 8 * B * c["T"],
                "flops": 16 * n}
    total = flops = 0
    for P, n in zip(*_lens(c)):
        tokens, pairs = P, n * P
        if op == "sparse_tree":
            keep = c["budget"] // 4 - 1
            common, runs = _windows(P // 4, keep, c["N"])
            runs = runs[:n]
            tokens = 4 * (common + _union(runs, P // 4 - common)) + P % 4
            pairs = sum(4 * (common + length) + P % 4 for _, length in runs)
            total += 4 * n * (keep + 1)
        total += (tokens + n) * c["Hkv"] * D * 4 + n * c["Hq"] * (4 * D + 4)
        flops += 4 * D * c["Hq"] * (pairs + n)
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------- exact --

def _wheel(x, pos, f, mscale, layout, sign):
    """The rotation as products of complex numbers, in 64 bits."""
    rot = 2 * f.numel()
    x = x.double()
    head, tail = x[..., :rot], x[..., rot:]
    pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if layout == "half" \
        else head.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_complex(pairs.contiguous())
    angle = sign * pos[..., None] * f
    y = torch.view_as_real(z * torch.polar(torch.full_like(angle, mscale), angle)[:, :, None])
    y = y.transpose(-1, -2).flatten(-2) if layout == "half" else y.flatten(-2)
    return torch.cat([y, tail], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    c, op = case, case["op"]
    if op == "rope":
        return {"y": _wheel(s["x"], s["pos"], s["freq"], s["mscale"], c["layout"],
                            -1.0 if c["transpose"] else 1.0)}
    if op in ("norm_rope", "norm_rope_grad"):
        unit = lambda x: x.double() / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt()
    if op == "norm_rope":
        turned = lambda x, w: _wheel(unit(x) * w.double(), s["pos"], s["freq"], s["mscale"],
                                     c["layout"], 1.0)
        kc, vc, k = s["k_cache"].double(), s["v_cache"].double(), turned(s["k"], s["k_weight"])
        for b in range(c["B"]):
            kc[b].index_copy_(0, s["slot"][b], k[b])
            vc[b].index_copy_(0, s["slot"][b], s["v"][b].double())
        return {"q": turned(s["q"], s["q_weight"]), "k_cache": kc, "v_cache": vc}
    if op == "norm_rope_grad":
        out = {}
        for n in "qk":
            x, w = s[n].double(), s[n + "_weight"].double()
            dz = _wheel(s["d_" + n], s["pos"], s["freq"], s["mscale"], c["layout"], -1.0)
            size = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            out["d%s_weight" % n] = torch.einsum("bthd,bthd->d", dz, x / size)
            along = (dz * w * x).sum(-1, keepdim=True) / (c["D"] * size.pow(3))
            out["d" + n] = dz * w / size - along * x
        return {n: out[n] for n in ("dq", "dk", "dq_weight", "dk_weight")}
    if work(case)["flops"] > 3e11:
        return None
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device=DEV)
    G = c["Hq"] // c["Hkv"]
    parents = s["parent"].tolist()
    for b, (P, n) in enumerate(zip(s["prefix"], s["drafts"])):
        seen = torch.zeros(n, P + n, dtype=torch.bool)
        if op == "dense_tree":
            seen[:, :P] = True
        else:
            seen[:, P // 4 * 4:P] = True
            for i, row in enumerate(s["sel"][b, :n].tolist()):
                blk = torch.tensor([j for j in row if 0 <= j < P // 4], dtype=torch.long)
                for k in range(4):
                    seen[i, blk * 4 + k] = True
        for i in range(n):
            j = i
            while j >= 0:
                seen[i, P + j] = True
                j = parents[b][j]
        seen = seen.to(DEV)
        for h in range(c["Hq"]):
            k, v = s["k_cache"][b, :P + n, h // G].double(), s["v_cache"][b, :P + n, h // G].double()
            x = (s["q"][b, :n, h].double() @ k.T / math.sqrt(c["D"])).where(seen, -math.inf)
            lse[b, :n, h] = torch.logsumexp(x, -1)
            o[b, :n, h] = torch.exp(x - lse[b, :n, h, None]) @ v
    return {"o": o, "lse": lse}
