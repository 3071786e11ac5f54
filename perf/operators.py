"""Cases of the tree-verify operators: what one pass of a drafted token tree through a model adds to the projections.

A step of tree-speculative decoding scores a small tree of drafted tokens in one pass: the projections' q, k and v rows
are normalised per head, rotated and appended to the cache (``append``); every node attends over the cached prefix and
its own ancestors (``attend``); the logits of every node get the sampling adjustments and a greedy choice (``adjust``);
the longest drafted path that agrees with the model is accepted and its cache rows become the sequence's (``accept``).

``run`` computes each in plain torch operations where ``own`` is false and calls the library where it is true;
``exact`` is the definition in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
QWORDS = 32  # bits per mask word


def _nt():
    from packed_weight_gemv_gb300 import nt
    return nt


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # one new token late in a 32K context, 8B-shaped heads, fp32 straight from the projections: pure latency
        dict(name="append_1", op="append", B=1, Hq=32, Hkv=8, D=128, rd=128, layout="half", dtype="f32", fused=True,
             tree=False, scaling="plain", pos0=31999, seed_rows=32768),
        # a drafted tree of 64 nodes, 16-bit activations, interleaved pairs over half of the head, a stretched context
        dict(name="append_tree_64", op="append", B=64, Hq=32, Hkv=8, D=128, rd=64, layout="interleaved", dtype="bf16",
             fused=False, tree=True, scaling="wavelength", pos0=90001, seed_rows=1024),
        # a prompt of 8,191 tokens, the projections' rows side by side in one buffer: bound by memory
        dict(name="append_prompt", op="append", B=8191, Hq=32, Hkv=8, D=128, rd=128, layout="half", dtype="f32",
             fused=True, tree=False, scaling="linear", pos0=0, seed_rows=8192),
        # a single token over a middling context (no drafts): the decode form
        dict(name="attend_1", op="attend", B=1, Hq=32, Hkv=8, D=128, dtype="f32", prefix=4095, gap=0),
        # a tree of 25 nodes at 26K tokens, fp32 queries as the append gives them
        dict(name="attend_25", op="attend", B=25, Hq=32, Hkv=8, D=128, dtype="f32", prefix=25999, gap=0),
        # a tree of 64 nodes kept in a scratch region behind the sequence's rows, 16-bit activations
        dict(name="attend_64_bf16", op="attend", B=64, Hq=32, Hkv=8, D=128, dtype="bf16", prefix=32704, gap=77),
        # a wide tree over narrow heads: products dominate
        dict(name="attend_255_narrow", op="attend", B=255, Hq=32, Hkv=4, D=64, dtype="f32", prefix=16001, gap=0),
        # one row of logits with every adjustment
        dict(name="adjust_1", op="adjust", B=1, V=151936, paths=False, mask="shared", bias=True, out=True),
        # a tree of 64 nodes: every node counts its own path and has its own grammar state
        dict(name="adjust_tree_64", op="adjust", B=64, V=151936, paths=True, mask="row", bias=True, out=True),
        # 16 nodes over an odd vocabulary, only the greedy token wanted
        dict(name="adjust_greedy_16", op="adjust", B=16, V=32003, paths=True, mask="row", bias=False, out=False),
        # a chain of 8 drafts, 5 accepted, 36 layers' caches
        dict(name="accept_chain_8", op="accept", B=8, L=36, Hkv=8, D=128, shape="chain", accepted=5, prefix=1023),
        # a wide tree with a long agreement
        dict(name="accept_tree_256", op="accept", B=256, L=36, Hkv=8, D=128, shape="tree", accepted=20, prefix=4000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "adjust", "accept"))
    if op == "append":
        D = rng.choice((64, 96, 128, 256))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 4, 7))
        B = _log(rng, 1, max(1, min(8191, 8191 * 48 * 128 // ((Hq + 2 * Hkv) * D))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, rd=rng.choice((D, D // 2, D // 4)),
                    layout=rng.choice(("half", "interleaved")), dtype=rng.choice(("f32", "bf16")),
                    fused=rng.random() < 0.5, tree=B <= 256 and rng.random() < 0.5,
                    scaling=rng.choice(("plain", "linear", "wavelength")), pos0=rng.randrange(0, 120000),
                    seed_rows=B + rng.randrange(0, 300))
    if op == "attend":
        D = rng.choice((64, 128))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 4, 5, 8))
        B = _log(rng, 1, 256)
        most = 255 * 16001 * 32 * 64 // (B * Hq * D)  # no more products than the largest listed case
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, dtype=rng.choice(("f32", "bf16")),
                    prefix=_log(rng, 1, max(1, min(32768, most))) if rng.random() < 0.95 else 0, gap=rng.choice((0, 0, 1, 200)))
    if op == "adjust":
        return dict(op=op, B=_log(rng, 1, 64), V=_log(rng, 1000, 151936), paths=rng.random() < 0.6,
                    mask=rng.choice(("none", "shared", "row")), bias=rng.random() < 0.5, out=rng.random() < 0.7)
    B = _log(rng, 2, 256)
    return dict(op=op, B=B, L=rng.randrange(1, 37), Hkv=rng.choice((1, 2, 4, 8)), D=rng.choice((64, 128)),
                shape=rng.choice(("chain", "tree")), accepted=rng.randrange(1, min(B, 24) + 1), prefix=rng.randrange(1, 4000))


# ---- inputs --------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g, np.random.RandomState(seed % (2 ** 32 - 1))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _parents(rs, B, shape="tree"):
    """Parent of each node (the root, node 0, has -1); always before the node itself."""
    if shape == "chain":
        return np.arange(-1, B - 1, dtype=np.int32)
    back = rs.randint(1, 9, B)
    return np.maximum(np.arange(B) - back, np.where(np.arange(B) == 0, -1, 0)).astype(np.int32)


def _ancestors(parent):
    """seen[b][j]: node j is b or one of its ancestors."""
    seen = np.eye(len(parent), dtype=bool)
    for b, p in enumerate(parent):
        if p >= 0:
            seen[b] |= seen[p]
    return seen


def _pack(bits):
    """Rows of truth values as int32 words, the lowest bit first."""
    rows, n = bits.shape
    words = (n + QWORDS - 1) // QWORDS
    full = np.zeros((rows, words * QWORDS), dtype=np.uint8)
    full[:, :n] = bits
    return torch.from_numpy(np.packbits(full, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)


def _frequencies(case):
    """Angle per position of each pair, in 64 bits (a model's constants)."""
    rd = case["rd"]
    f = 1e6 ** (-2.0 * torch.arange(rd // 2, dtype=torch.float64, device=DEV) / rd)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "wavelength":
        turns = 32768.0 * f / (2.0 * math.pi)
        w = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * (w + (1.0 - w) / 4.0), 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    g, rs = _gen(seed)
    s = dict(case=case)
    B = case["B"]
    if case["op"] == "append":
        Hq, Hkv, D, t = case["Hq"], case["Hkv"], case["D"], _dtype(case)
        if case["fused"]:  # one projection buffer per token: q, k and v heads side by side
            qkv = (_normal(g, B, Hq + 2 * Hkv, D) * 1.7).to(t)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = ((_normal(g, B, h, D) * 1.7).to(t) for h in (Hq, Hkv, Hkv))
        s["q_gamma"], s["k_gamma"] = 1.0 + 0.2 * _normal(g, D), 1.0 + 0.2 * _normal(g, D)
        s["inv_freq"], s["amplitude"] = _frequencies(case)
        s["pos"] = None
        if case["tree"]:
            s["pos"] = torch.from_numpy((_ancestors(_parents(rs, B)).sum(1) - 1 + case["pos0"]).astype(np.int32)).to(DEV)
        rows = max(case["seed_rows"], B)
        s["row0"] = rows - B
        s["k_cache"] = torch.zeros(Hkv, rows, D, dtype=torch.bfloat16, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["q_out"] = torch.empty(B, Hq, D, dtype=t, device=DEV)
    elif case["op"] == "attend":
        Hq, Hkv, D, t = case["Hq"], case["Hkv"], case["D"], _dtype(case)
        s["row0"] = case["prefix"] + case["gap"]
        rows = s["row0"] + B
        s["q"] = (_normal(g, B, Hq, D) * 1.5).to(t)
        s["k_cache"] = _normal(g, Hkv, rows, D).bfloat16()
        s["v_cache"] = _normal(g, Hkv, rows, D).bfloat16()
        s["mask"] = _pack(_ancestors(_parents(rs, B)))
        s["out"] = torch.empty(B, Hq, D, dtype=t, device=DEV)
        if own:
            nt = _nt()
            s["ws"] = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hq, Hkv, D, case["prefix"]), dtype=torch.uint8, device=DEV)
    elif case["op"] == "adjust":
        V = case["V"]
        s["logits"] = _normal(g, B, V) * 3.0
        # tokens of the context so far: a long tail of single uses, a few that come often
        seen = (torch.rand(4096, generator=g, device=DEV) ** 3 * V).long().clamp(max=V - 1)
        s["counts"] = torch.zeros(V, dtype=torch.int32, device=DEV).index_add_(0, seen, torch.ones_like(seen, dtype=torch.int32))
        s["tree_mask"] = s["tokens"] = None
        if case["paths"]:
            s["tree_mask"] = _pack(_ancestors(_parents(rs, B)))
            s["tokens"] = torch.from_numpy(rs.randint(0, V, B).astype(np.int32)).to(DEV)
        s["bias"] = None
        if case["bias"]:
            s["bias"] = torch.where(torch.rand(V, generator=g, device=DEV) < 0.01, 4.0 * _normal(g, V), torch.zeros(V, device=DEV))
        s["allowed"] = None
        if case["mask"] != "none":  # a grammar's states allow anything from half of the tokens to a handful
            rows = 1 if case["mask"] == "shared" else B
            share = torch.pow(10.0, -3.0 * torch.rand(rows, 1, generator=g, device=DEV)) * 0.5
            words = (V + QWORDS - 1) // QWORDS
            bits = torch.rand(rows, words * QWORDS, generator=g, device=DEV) < share
            weight = torch.tensor([1 << i for i in range(31)] + [-(1 << 31)], dtype=torch.int64, device=DEV)
            s["allowed"] = (bits.view(rows, words, QWORDS).long() * weight).sum(2).int()
        s["out"] = torch.empty(B, V, device=DEV) if case["out"] else None
        s["argmax"] = torch.empty(B, dtype=torch.int32, device=DEV)
        if own:
            s["ws"] = torch.zeros(_nt().nt_logits_adjust_workspace_size(V, B), dtype=torch.uint8, device=DEV)
    else:
        L, Hkv, D, P = case["L"], case["Hkv"], case["D"], case["prefix"]
        parent = _parents(rs, B, case["shape"])
        anc = _ancestors(parent)
        token = rs.randint(0, 151936, B).astype(np.int32)
        choice = rs.randint(0, 151936, B).astype(np.int32)
        depth = anc.sum(1)
        deep = np.flatnonzero(depth == min(case["accepted"], depth.max()))
        path = np.flatnonzero(anc[deep[rs.randint(len(deep))]])  # the agreed path, root first
        choice[path[:-1]] = token[path[1:]]
        s["parent"], s["token"], s["choice"] = (torch.from_numpy(a).to(DEV) for a in (parent, token, choice))
        s["anc"] = torch.from_numpy(anc).to(DEV)
        s["row0"] = P + B  # the tree's rows stand behind a region that the accepted ones move into
        s["cache"] = _normal(g, L, 2, Hkv, P + 2 * B, D).bfloat16()
        s["emit"], s["path"] = (torch.empty(B, dtype=torch.int32, device=DEV) for _ in range(2))
        s["n"] = torch.empty(1, dtype=torch.int32, device=DEV)
        if own:
            nt = _nt()
            s["k_caches"], s["v_caches"] = (nt.pointer_array([s["cache"][i, j] for i in range(L)]) for j in range(2))
    return s


# ---- one pass ------------------------------------------------------------------------------
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
EPS = 1e-6
REPETITION, FREQUENCY, PRESENCE = 1.1, 0.3, 0.2


def _rotate(x, gamma, angle_cos, angle_sin, layout):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma
    h = angle_cos.shape[-1]
    c, d = angle_cos[:, None, :], angle_sin[:, None, :]
    if layout == "half":
        a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
        return torch.cat((a * c - b * d, b * c + a * d, rest), -1)
    a, b, rest = x[..., 0:2 * h:2], x[..., 1:2 * h:2], x[..., 2 * h:]
    return torch.cat((torch.stack((a * c - b * d, b * c + a * d), -1).flatten(-2), rest), -1)


def _append(s):
    case = s["case"]
    B, r0 = case["B"], s["row0"]
    pos = s["pos"] if s["pos"] is not None else case["pos0"] + torch.arange(B, device=DEV)
    angle = pos.double()[:, None] * s["inv_freq"][None, :]
    c, d = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    s["q_out"].copy_(_rotate(s["q"], s["q_gamma"], c, d, case["layout"]))
    s["k_cache"][:, r0:r0 + B] = _rotate(s["k"], s["k_gamma"], c, d, case["layout"]).transpose(0, 1).bfloat16()
    s["v_cache"][:, r0:r0 + B] = s["v"].float().transpose(0, 1).bfloat16()
    return s["q_out"]


def _bits(words, n):
    b = (words[:, :, None] >> torch.arange(QWORDS, device=DEV, dtype=torch.int32)) & 1
    return b.reshape(words.shape[0], -1)[:, :n].bool()


def _attend(s):
    case = s["case"]
    B, Hq, Hkv, D, P, r0 = case["B"], case["Hq"], case["Hkv"], case["D"], case["prefix"], s["row0"]
    G = Hq // Hkv
    k = torch.cat((s["k_cache"][:, :P], s["k_cache"][:, r0:r0 + B]), 1).float()
    v = torch.cat((s["v_cache"][:, :P], s["v_cache"][:, r0:r0 + B]), 1).float()
    q = s["q"].float().view(B, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * B, D)
    w = torch.matmul(q, k.transpose(1, 2)).view(Hkv, G, B, P + B) * (1.0 / math.sqrt(D))
    w[..., P:].masked_fill_(~_bits(s["mask"], B), -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    out = torch.matmul(w.view(Hkv, G * B, P + B), v).view(Hkv, G, B, D) / w.sum(-1, keepdim=True)
    s["out"].copy_(out.permute(2, 0, 1, 3).reshape(B, Hq, D))
    return s["out"]


def _adjust(s):
    case = s["case"]
    B, V = case["B"], case["V"]
    count = s["counts"].expand(B, V)
    if s["tokens"] is not None:
        seen = _bits(s["tree_mask"], B).int()
        count = count + torch.zeros(B, V, dtype=torch.int32, device=DEV).index_add_(1, s["tokens"].long(), seen)
    x, c = s["logits"], count.float()
    y = torch.where(x > 0, x / REPETITION, x * REPETITION)
    y = torch.where(count > 0, (y - FREQUENCY * c) - PRESENCE, x)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["allowed"] is not None:
        y = y.masked_fill(~_bits(s["allowed"], V), -math.inf)
    best = y.amax(-1, keepdim=True)
    at = torch.where(y == best, torch.arange(V, device=DEV), V).amin(-1)
    s["argmax"].copy_(torch.where(best[:, 0] > -math.inf, at, -1))
    if s["out"] is not None:
        s["out"].copy_(y)
    return s["out"], s["argmax"]


def _accept(s):
    case = s["case"]
    B, P, r0 = case["B"], case["prefix"], s["row0"]
    node = torch.arange(B, device=DEV)
    up = s["parent"].clamp(min=0).long()
    match = (s["token"] == s["choice"][up]) & (s["parent"] >= 0)
    twin = (s["parent"][:, None] == s["parent"][None, :]) & match[None, :] & (node[None, :] < node[:, None])
    ok = (match & ~twin.any(1)) | (node == 0)
    taken = ~(s["anc"] & ~ok[None, :]).any(1)
    n = taken.sum()
    slot = torch.where(taken, taken.cumsum(0) - 1, B)
    path = torch.full((B + 1,), -1, dtype=torch.int32, device=DEV).scatter_(0, slot, node.int())[:B]
    s["path"].copy_(path)
    s["emit"].copy_(torch.where(node < n, s["choice"][path.clamp(min=0).long()], -1))
    s["n"].copy_(n)
    moved = s["cache"][:, :, :, r0 + path.clamp(min=0).long()]
    into = s["cache"][:, :, :, P:P + B]
    into.copy_(torch.where((node < n)[:, None], moved, into))
    return s["emit"], s["path"], s["n"], into


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "append":
        r0, B = s["row0"], case["B"]
        if own:
            _nt().nt_qk_norm_rope_append(s["q"], s["k"], s["v"], s["q_gamma"], s["k_gamma"], EPS, s["inv_freq"],
                                         ROPE_LAYOUTS[case["layout"]], s["amplitude"], s["q_out"], s["k_cache"],
                                         s["v_cache"], pos=s["pos"], pos0=case["pos0"], row0=r0)
        else:
            _append(s)
        return s["q_out"], s["k_cache"][:, r0:r0 + B], s["v_cache"][:, r0:r0 + B]
    if op == "attend":
        if not own:
            return _attend(s)
        _nt().nt_tree_attention(s["q"], s["k_cache"], s["v_cache"], case["prefix"], s["row0"], s["mask"], s["out"], s["ws"])
        return s["out"]
    if op == "adjust":
        if not own:
            return _adjust(s)
        _nt().nt_logits_adjust(s["logits"], counts=s["counts"], tree_mask=s["tree_mask"], tokens=s["tokens"],
                               repetition=REPETITION, frequency=FREQUENCY, presence=PRESENCE, bias=s["bias"],
                               allowed=s["allowed"], out=s["out"], argmax=s["argmax"], ws=s["ws"])
        return s["out"], s["argmax"]
    if not own:
        return _accept(s)
    nt, P, B = _nt(), case["prefix"], case["B"]
    nt.nt_tree_accept(s["parent"], s["token"], s["choice"], s["emit"], s["path"], s["n"])
    nt.nt_tree_commit(s["k_caches"], s["v_caches"], case["Hkv"], case["D"], P + 2 * B, s["path"], s["n"], s["row0"], P)
    return s["emit"], s["path"], s["n"], s["cache"][:, :, :, P:P + B]


# ---- cost and definition -------------------------------------------------------------------
def work(case):
    B = case["B"]
    if case["op"] == "append":
        size = 4 if case["dtype"] == "f32" else 2
        rows_in, rows_q, rows_c = case["Hq"] + 2 * case["Hkv"], case["Hq"], 2 * case["Hkv"]
        D = case["D"]
        return dict(bytes=B * D * (size * (rows_in + rows_q) + 2 * rows_c) + 4 * case["rd"] + 8 * D + (4 * B if case["tree"] else 0),
                    flops=B * D * (case["Hq"] + case["Hkv"]) * 7)
    if case["op"] == "attend":
        size = 4 if case["dtype"] == "f32" else 2
        keys = case["prefix"] + B
        return dict(bytes=2 * 2 * case["Hkv"] * keys * case["D"] + 2 * size * B * case["Hq"] * case["D"] + B * ((B + 31) // 32) * 4,
                    flops=4 * B * case["prefix"] * case["Hq"] * case["D"] + 4 * case["Hq"] * case["D"] * B)
    if case["op"] == "adjust":
        V = case["V"]
        masks = {"none": 0, "shared": 1, "row": B}[case["mask"]]
        return dict(bytes=4 * B * V * (2 if case["out"] else 1) + 4 * V * (2 if case["bias"] else 1) + masks * ((V + 31) // 32) * 4 + 4 * B,
                    flops=6 * B * V)
    rows = min(case["accepted"], B)
    return dict(bytes=2 * rows * case["L"] * 2 * case["Hkv"] * case["D"] * 2 + 5 * 4 * B, flops=B * rows)


def _exact_append(s):
    case = s["case"]
    B, rd = case["B"], case["rd"]
    pos = np.arange(B) + case["pos0"] if s["pos"] is None else s["pos"].cpu().numpy()
    theta = torch.from_numpy(pos.astype(np.float64)).to(DEV).outer(s["inv_freq"])
    turn = torch.polar(torch.full_like(theta, s["amplitude"]), theta)[:, None, :]  # complex: a rotation is one product

    def head(x, gamma):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gamma.double()
        first, second = (slice(0, rd // 2), slice(rd // 2, rd)) if case["layout"] == "half" else (slice(0, rd, 2), slice(1, rd, 2))
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    return head(s["q"], s["q_gamma"]), head(s["k"], s["k_gamma"]).transpose(0, 1), s["v"].double().transpose(0, 1)


def _exact_attend(s):
    case = s["case"]
    B, Hq, P, r0 = case["B"], case["Hq"], case["prefix"], s["row0"]
    words = s["mask"].cpu().numpy().view(np.uint32)
    sees = torch.tensor([[bool(words[b, j // 32] >> (j % 32) & 1) for j in range(B)] for b in range(B)], device=DEV)
    out = torch.zeros(B, Hq, case["D"], dtype=torch.float64, device=DEV)
    for h in range(Hq):
        g = h * case["Hkv"] // Hq
        score = s["q"][:, h].double() @ s["k_cache"][g].double().T / case["D"] ** 0.5
        score[:, P:r0] = -math.inf
        score[:, r0:][~sees] = -math.inf
        out[:, h] = score.softmax(-1) @ s["v_cache"][g].double()
    return out


def _exact_adjust(s):
    case = s["case"]
    x = s["logits"].cpu().numpy().astype(np.float64)
    B, V = x.shape
    counts = np.tile(s["counts"].cpu().numpy().astype(np.int64), (B, 1))
    if s["tokens"] is not None:
        words, tokens = s["tree_mask"].cpu().numpy().view(np.uint32), s["tokens"].cpu().numpy()
        for b in range(B):
            for j in range(B):
                counts[b, tokens[j]] += int(words[b, j // 32] >> (j % 32) & 1)
    used = counts > 0
    x[used] = np.where(x[used] > 0, x[used] / REPETITION, x[used] * REPETITION) - FREQUENCY * counts[used] - PRESENCE
    if s["bias"] is not None:
        x += s["bias"].cpu().numpy()
    if s["allowed"] is not None:
        bits = np.unpackbits(s["allowed"].cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :V]
        x[~np.broadcast_to(bits.astype(bool), x.shape)] = -np.inf
    return torch.from_numpy(x), None  # the choice is a whole number: near ties go by the 32-bit values


def _exact_accept(s):
    case = s["case"]
    parent, token, choice = (s[k].tolist() for k in ("parent", "token", "choice"))
    path = [0]
    while True:
        agreed = [c for c in range(case["B"]) if parent[c] == path[-1] and token[c] == choice[path[-1]]]
        if not agreed:
            break
        path.append(agreed[0])
    rows = s["cache"].double()[:, :, :, case["prefix"]:case["prefix"] + case["B"]].clone()
    for i, node in enumerate(path):
        rows[:, :, :, i] = s["cache"][:, :, :, s["row0"] + node]
    return None, None, None, rows


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "adjust":
        return _exact_adjust(s) if case["out"] else None  # a lone choice has no 64-bit value
    return _exact_accept(s)
