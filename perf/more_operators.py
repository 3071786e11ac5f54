"""Cases of the paged-cache operators: what serving several sequences, and beams of them, adds to the projections.

A pool holds the cached keys and values of all sequences in pages of a few rows; a table names the pages of each sequence,
and pages that several sequences share are counted. A step attends with ragged chunks of new tokens over the pages
(``attend``: prompts, chunks of prompts and single tokens alike), chooses the next beams over beams and vocabulary
(``beam``), and lets the tables follow them: sequences are forked, dropped and extended, shared pages are copied
before they are written (``pages``). Now and then the pool is compacted (``compact``).

``run`` computes each in plain torch operations where ``own`` is false and calls the library where it is true;
``exact`` is the definition in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def _nt():
    from packed_weight_gemv_gb300 import nt
    return nt


# ---- cases ---------------------------------------------------------------------------------
# An attention case lists its sequences as "new+before" (new tokens, rows cached before them).
def listed():
    return [
        # one new token late in a 4K context, 8B-shaped heads, fp32 straight from the projections: pure latency
        dict(name="attend_token", op="attend", seqs="1+4094", Hq=32, Hkv=8, D=128, page=16, dtype="f32", window=0, cap=0.0,
             slopes=False),
        # 64 sequences of a serving batch decode one token each over 100 to 12,000 rows: bound by memory
        dict(name="attend_batch_64", op="attend", seqs=_spread(64, 100, 12000), Hq=32, Hkv=8, D=128, page=16, dtype="f32",
             window=0, cap=0.0, slopes=False),
        # a chunk of a long prompt, fp32 straight from the projections: bound by products
        dict(name="attend_chunk_511", op="attend", seqs="511+7489", Hq=32, Hkv=8, D=128, page=64, dtype="f32", window=0,
             cap=0.0, slopes=False),
        # whole prompts of ragged lengths in one pass, 16-bit activations
        dict(name="attend_prompts", op="attend", seqs="4001+0 77+0 2049+16000 1+0 1900+301", Hq=32, Hkv=8, D=128, page=32,
             dtype="bf16", window=0, cap=0.0, slopes=False),
        # a chunk among 40 decoding sequences: capped scores, distance bias and a window, narrow heads
        dict(name="attend_mixed_capped", op="attend", seqs="257+9000 " + _spread(40, 30, 6000), Hq=32, Hkv=4, D=64, page=128,
             dtype="bf16", window=4096, cap=30.0, slopes=True),
        # four beams of one request over the whole vocabulary
        dict(name="beam_4", op="beam", groups=1, W=4, K=4, V=151936, done=0.0, alpha=0.0),
        # 16 requests of 8 beams: bound by reading the logits
        dict(name="beam_16x8", op="beam", groups=16, W=8, K=8, V=151936, done=0.2, alpha=0.6),
        # an odd vocabulary, twice as many candidates as beams
        dict(name="beam_3x16_odd", op="beam", groups=3, W=16, K=32, V=32003, done=0.1, alpha=0.0),
        # the next step of 8 beams of one request, 36 layers: latency
        dict(name="pages_beam_8", op="pages", groups=1, W=8, L=36, Hkv=8, D=128, page=16, prompt=1000, since=21, new=1, drop=0.0),
        # the next step of 32 requests of 8 beams, some of them finished
        dict(name="pages_32x8", op="pages", groups=32, W=8, L=4, Hkv=8, D=128, page=16, prompt=700, since=60, new=1, drop=0.1),
        # a small pool after some sequences have gone
        dict(name="compact_300", op="compact", pages=300, S=5, L=6, Hkv=8, D=128, page=16, used=0.4),
        # a large one: bound by moving the pages
        dict(name="compact_6000", op="compact", pages=6000, S=100, L=2, Hkv=8, D=128, page=16, used=0.6),
    ]


def _spread(n, lo, hi):
    """n decoding sequences, their lengths spread over their logarithm."""
    return " ".join(f"1+{int(lo * (hi / lo) ** (((i * 29) % n + 0.5) / n))}" for i in range(n))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sequences(case):
    return [tuple(int(x) for x in s.split("+")) for s in case["seqs"].split()]


def draw(rng):
    op = rng.choice(("attend", "attend", "beam", "pages", "compact"))
    if op == "attend":
        D = rng.choice((64, 128))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 4, 5, 8))
        seqs, rows, products = [], 150000, 2049 * 17000 * 32 * 128  # no more than the largest listed cases
        for _ in range(_log(rng, 1, 64)):
            before = 0 if rng.random() < 0.1 else _log(rng, 1, 16000)
            most = min(2048, products // (2 * Hq * D * (before + 1024)))
            new = 1 if rng.random() < 0.6 else _log(rng, 1, max(1, most))
            rows -= new + before
            products -= new * (before + (new + 1) // 2) * Hq * D
            if seqs and (rows < 0 or products < 0):
                break
            seqs.append(f"{new}+{before}")
        return dict(op=op, seqs=" ".join(seqs), Hq=Hq, Hkv=Hkv, D=D, page=rng.choice((16, 32, 64, 128, 256)),
                    dtype=rng.choice(("f32", "bf16")), window=rng.choice((0, 0, _log(rng, 1, 8192))),
                    cap=rng.choice((0.0, 0.0, 30.0, 50.0)), slopes=rng.random() < 0.25)
    if op == "beam":
        W = _log(rng, 1, 32)
        return dict(op=op, groups=_log(rng, 1, max(1, 128 // W)), W=W, K=min(64, W * rng.choice((1, 1, 2))),
                    V=_log(rng, 1000, 151936), done=rng.choice((0.0, 0.2)), alpha=rng.choice((0.0, 0.6, 1.0)))
    if op == "pages":
        return dict(op=op, groups=_log(rng, 1, 32), W=_log(rng, 1, 8), L=rng.randrange(1, 5), Hkv=rng.choice((1, 2, 4, 8)),
                    D=rng.choice((64, 128)), page=rng.choice((16, 32)), prompt=_log(rng, 1, 700), since=rng.randrange(0, 70),
                    new=rng.choice((1, 1, 3)), drop=rng.choice((0.0, 0.2)))
    return dict(op=op, pages=_log(rng, 50, 6000), S=_log(rng, 1, 100), L=rng.randrange(1, 3), Hkv=rng.choice((1, 2, 4, 8)),
                D=rng.choice((64, 128)), page=16, used=rng.uniform(0.1, 0.95))


# ---- inputs --------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g, np.random.RandomState(seed % (2 ** 32 - 1))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _uneven(n):
    """n numbers in [0, 1), spread unevenly: the sizes of a case do not depend on the seed."""
    return (0.3 + np.arange(n) * 0.6180339887498949) % 1.0


def _start(counts):
    return np.concatenate(([0], np.cumsum(counts)))


def _prepare_attend(case, g, rs, s):
    Hq, Hkv, D, page, t = case["Hq"], case["Hkv"], case["D"], case["page"], _dtype(case)
    new, before = (np.array(x) for x in zip(*_sequences(case)))
    length, S = new + before, len(new)
    held = -(-length // page)
    n_pages = int(held.sum()) + 7
    ids, table = rs.permutation(n_pages), np.full((S, int(held.max()) + 1), -1)
    for i, at in enumerate(_start(held)[:-1]):
        table[i, :held[i]] = ids[at:at + held[i]]
    s["new"], s["seen"] = new.tolist(), length.tolist()
    s["table"], s["length"], s["q_start"] = _ints(table), _ints(length), _ints(_start(new))
    s["q"] = (_normal(g, int(new.sum()), Hq, D) * 1.5).to(t)
    s["k_pool"], s["v_pool"] = (_normal(g, Hkv, n_pages * page, D).bfloat16() for _ in range(2))
    s["slopes"] = None
    if case["slopes"]:
        s["slopes"] = torch.pow(2.0, -8.0 * (torch.arange(Hq, device=DEV) + 1.0) / Hq)
    s["out"] = torch.empty_like(s["q"])
    if own:
        nt = _nt()
        s["ws"] = torch.zeros(nt.nt_paged_attention_workspace_size(int(new.sum()), S, Hq, Hkv, D), dtype=torch.uint8, device=DEV)


def _prepare_beam(case, g, rs, s):
    G, W, K, V = case["groups"], case["W"], case["K"], case["V"]
    n = G * W
    # a peaked distribution over a flat tail, the peaks elsewhere in each row
    s["logits"] = _normal(g, n, V) * 2.0
    peaks = (torch.randint(0, V, (n, 1), generator=g, device=DEV) + torch.arange(12, device=DEV) * (V // 13)) % V
    s["logits"].scatter_add_(1, peaks, 6.0 + 3.0 * torch.rand(n, 12, generator=g, device=DEV))
    s["scores"] = -12.0 * torch.rand(n, generator=g, device=DEV)
    s["done"] = (torch.rand(n, generator=g, device=DEV) < case["done"]).int()
    s["lengths"] = torch.randint(1, 40, (n,), generator=g, device=DEV, dtype=torch.int32)
    s["eos"] = V - 2
    s["parent"], s["token"], s["done_out"] = (torch.empty(G * K, dtype=torch.int32, device=DEV) for _ in range(3))
    s["score"] = torch.empty(G * K, device=DEV)
    if own:
        s["ws"] = torch.zeros(_nt().nt_beam_select_workspace_size(V, n), dtype=torch.uint8, device=DEV)


def _prepare_pages(case, g, rs, s):
    G, W, page, new = case["groups"], case["W"], case["page"], case["new"]
    S = G * W
    prompt = np.maximum(1, (case["prompt"] * (0.6 + 0.8 * _uneven(G))).astype(np.int64))
    shared = prompt // page  # whole pages of the prompt stand once; the rest of each beam is its own
    length = np.repeat(prompt + case["since"], W)
    held = -(-length // page)
    width = int(held.max()) + 2 + new // page
    table = np.full((S, width), -1)
    ids = rs.permutation(int(shared.sum() + (held - np.repeat(shared, W)).sum()))
    at = 0
    for i in range(G):
        table[i * W:(i + 1) * W, :shared[i]] = ids[at:at + shared[i]]
        at += shared[i]
        for j in range(i * W, (i + 1) * W):
            table[j, shared[i]:held[j]] = ids[at:at + held[j] - shared[i]]
            at += held[j] - shared[i]
    n_used = len(ids)
    n_pages = n_used + S * (2 + new // page)
    refs = np.bincount(table[table >= 0], minlength=n_pages)
    parent = np.repeat(np.arange(G) * W, W) + (rs.uniform(0, 1, S) ** 2 * W).astype(np.int64)  # the better beams have more children
    parent[rs.uniform(0, 1, S) < case["drop"]] = -1
    s["width"] = width
    s["table"], s["length"], s["refs_before"], s["parent"] = _ints(table), _ints(length), _ints(refs), _ints(parent)
    s["refs"] = s["refs_before"].clone()
    s["table_out"], s["length_out"] = torch.empty_like(s["table"]), torch.empty_like(s["length"])
    s["q_start"] = _ints(np.arange(S + 1) * new)
    s["rows"], s["pos"] = (torch.empty(S * new, dtype=torch.int32, device=DEV) for _ in range(2))
    s["pairs"] = torch.empty(S, 2, dtype=torch.int32, device=DEV)
    _prepare_pool(case, g, s, n_pages)


def _prepare_compact(case, g, rs, s):
    n, S, page = case["pages"], case["S"], case["page"]
    used = max(1, int(n * case["used"]))
    ids = rs.permutation(n)[:used]
    held = np.diff(np.round(_start(0.1 + _uneven(S)) * used / (0.1 + _uneven(S)).sum()).astype(np.int64))
    table = np.full((S, int(held.max()) + 1), -1)
    for i, at in enumerate(_start(held)[:-1]):
        table[i, :held[i]] = ids[at:at + held[i]]
    if S > 1:  # some share the beginning of the one before
        for i in range(1, S, 3):
            both = min(held[i], held[i - 1]) // 2
            table[i, :both] = table[i - 1, :both]
    length = np.maximum(0, held * page - rs.randint(0, page, S))
    s["table_before"], s["length"] = _ints(table), _ints(length)
    s["refs_before"] = _ints(np.bincount(table[table >= 0], minlength=n))
    s["table"], s["refs"] = s["table_before"].clone(), s["refs_before"].clone()
    s["pairs"] = torch.empty(n // 2, 2, dtype=torch.int32, device=DEV)
    s["n_used"] = torch.empty(1, dtype=torch.int32, device=DEV)
    _prepare_pool(case, g, s, n)
    if own:
        s["ws"] = torch.zeros(_nt().nt_page_compact_workspace_size(n), dtype=torch.uint8, device=DEV)


def _prepare_pool(case, g, s, n_pages):
    L = case["L"]
    s["cache"] = _normal(g, L, 2, case["Hkv"], n_pages * case["page"], case["D"]).bfloat16()
    if own:
        s["k_caches"], s["v_caches"] = (_nt().pointer_array([s["cache"][i, j] for i in range(L)]) for j in range(2))


def prepare(case, seed):
    g, rs = _gen(seed)
    s = dict(case=case)
    {"attend": _prepare_attend, "beam": _prepare_beam, "pages": _prepare_pages, "compact": _prepare_compact}[case["op"]](case, g, rs, s)
    return s


# ---- one pass ------------------------------------------------------------------------------
def _pool_rows(pages, page):
    return (pages.long()[:, None] * page + torch.arange(page, device=DEV)).flatten()


def _attend(s):
    case = s["case"]
    Hq, Hkv, D, page, window, cap = case["Hq"], case["Hkv"], case["D"], case["page"], case["window"], case["cap"]
    G, at = Hq // Hkv, 0
    for i, (n, seen) in enumerate(zip(s["new"], s["seen"])):
        rows = _pool_rows(s["table"][i, :-(-seen // page)], page)[:seen]
        k, v = s["k_pool"][:, rows].float(), s["v_pool"][:, rows].float()
        block = max(1, (1 << 28) // (seen * Hq))  # queries at a time
        for a in range(0, n, block):
            b = min(n, a + block)
            q = s["q"][at + a:at + b].float().view(b - a, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * (b - a), D)
            w = torch.matmul(q, k.transpose(1, 2)).view(Hkv, G, b - a, seen) * (1.0 / math.sqrt(D))
            if cap > 0:
                w = cap * torch.tanh(w / cap)
            back = (seen - n + torch.arange(a, b, device=DEV))[:, None] - torch.arange(seen, device=DEV)  # distance to each row
            if s["slopes"] is not None:
                w = w - s["slopes"].view(Hkv, G, 1, 1) * back.float()
            w = w.masked_fill((back < 0) | (back >= window) if window > 0 else back < 0, -math.inf)
            w = torch.exp(w - w.amax(-1, keepdim=True))
            out = torch.matmul(w.view(Hkv, G * (b - a), seen), v).view(Hkv, G, b - a, D) / w.sum(-1, keepdim=True)
            s["out"][at + a:at + b] = out.permute(2, 0, 1, 3).reshape(b - a, Hq, D)
        at += n
    return s["out"]


def _beam(s):
    case = s["case"]
    G, W, K, V = case["groups"], case["W"], case["K"], case["V"]
    x, score = s["logits"].double(), s["scores"].double()[:, None]  # 64 bits: the order of values next to each other
    most = x.amax(-1, keepdim=True)
    total = score + (x - (most + (x - most).exp().sum(-1, keepdim=True).log()))
    done = s["done"][:, None] > 0
    only = torch.arange(V, device=DEV)[None, :] == s["eos"]
    total = torch.where(done, torch.where(only, score, -math.inf), total)
    length = (s["lengths"] + 1 - s["done"]).double()[:, None]
    rank, order = torch.sort((total / length ** case["alpha"]).view(G, W * V), dim=-1, descending=True, stable=True)
    rank, order = rank[:, :K], order[:, :K]
    there = rank > -math.inf
    beam = torch.arange(G, device=DEV)[:, None] * W + order // V
    token = order % V
    s["parent"].copy_(torch.where(there, beam, -1).flatten())
    s["token"].copy_(torch.where(there, token, -1).flatten())
    s["score"].copy_(torch.where(there, total.view(G, W * V).gather(1, order), -math.inf).flatten())
    s["done_out"].copy_((there & ((token == s["eos"]) | (s["done"][beam] > 0))).int().flatten())
    return s["parent"], s["token"], s["score"], s["done_out"]


def _counted(refs, table, length, page, sign):
    used = torch.arange(table.shape[1], device=DEV)[None, :] * page < length[:, None]
    refs.index_add_(0, torch.where(used, table, 0).flatten().long(), sign * used.flatten().int())
    return used


def _pages(s):
    case = s["case"]
    S, page, new, width = case["groups"] * case["W"], case["page"], case["new"], s["width"]
    refs, table, length = s["refs"], s["table_out"], s["length_out"]
    refs.copy_(s["refs_before"])
    # fork: every sequence goes on as its parent
    _counted(refs, s["table"], s["length"], page, -1)
    up = s["parent"].clamp(min=0).long()
    length.copy_(torch.where(s["parent"] >= 0, s["length"][up], 0))
    table.copy_(torch.where(torch.arange(width, device=DEV)[None, :] * page < length[:, None], s["table"][up], -1))
    _counted(refs, table, length, page, 1)
    # extend: the last page is given up where another sequence still holds it, and new ones are taken, lowest first
    last = (length - 1).clamp(min=0) // page
    holds = torch.where(length % page != 0, table.gather(1, last[:, None].long())[:, 0], -1)
    before = torch.tril(holds[:, None] == holds[None, :], -1).sum(1)  # sequences before this one with the same last page
    cow = ((holds >= 0) & (refs[holds.clamp(min=0).long()] - before > 1)).int()
    old, need = -(-length // page), -(-(length + new) // page)
    demand = need - old + cow
    upto = demand.cumsum(0)
    free = torch.where(refs == 0, torch.arange(len(refs), device=DEV), len(refs)).sort().values.int()
    column = torch.arange(width, device=DEV)[None, :]
    fresh = (column >= (old - cow)[:, None]) & (column < need[:, None])
    which = (upto - demand)[:, None] + column - (old - cow)[:, None]
    s["pairs"].copy_(torch.where(cow[:, None] > 0, torch.stack((holds, free[(upto - demand).long().clamp(max=len(free) - 1)]), 1), -1))
    table.copy_(torch.where(fresh, free[which.clamp(0, len(free) - 1).long()], table))
    refs.index_add_(0, holds.clamp(min=0).long(), -cow)
    refs.index_add_(0, torch.where(fresh, table, 0).flatten().long(), fresh.flatten().int())
    pos = (length[:, None] + torch.arange(new, device=DEV)).int()
    s["pos"].copy_(pos.flatten())
    s["rows"].copy_((table.gather(1, (pos // page).long()) * page + pos % page).flatten())
    length += new
    # copy: the shared pages that are about to be written, in every layer
    _copy(s["cache"], s["pairs"], page)
    return refs, table, length, s["rows"], s["pos"], s["pairs"], s["cache"]


def _copy(cache, pairs, page):
    there = pairs[:, :1] >= 0
    some = pairs[there[:, 0].int().argmax()].clamp(min=0)  # in place of a pair that is none: one that is (or page 0 onto itself)
    pairs = torch.where(there, pairs, some)
    cache[:, :, :, _pool_rows(pairs[:, 1], page)] = cache[:, :, :, _pool_rows(pairs[:, 0], page)]


def _compact(s):
    case = s["case"]
    n, page = case["pages"], case["page"]
    s["table"].copy_(s["table_before"])
    s["refs"].copy_(s["refs_before"])
    used = s["refs"] > 0
    count, page_id = used.sum(), torch.arange(n, device=DEV)
    source = torch.where(used & (page_id >= count), page_id, n).sort().values[:n // 2]
    into = torch.where(~used & (page_id < count), page_id, n).sort().values[:n // 2]
    moves = source < n
    s["pairs"].copy_(torch.where(moves[:, None], torch.stack((source, into), 1), -1))
    to = torch.arange(n + 1, device=DEV).scatter_(0, source, torch.where(moves, into, n))
    s["n_used"].copy_(count)
    held = torch.arange(s["table"].shape[1], device=DEV)[None, :] * page < s["length"][:, None]
    s["table"].copy_(torch.where(held, to[s["table"].clamp(min=0).long()], s["table"]))
    s["refs"].copy_(torch.zeros_like(s["refs"]).index_add_(0, to[:n], s["refs"]))
    _copy(s["cache"], s["pairs"], page)
    return s["refs"], s["table"], s["pairs"], s["n_used"], s["cache"]


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "attend":
        if not own:
            return _attend(s)
        _nt().nt_paged_attention(s["q"], s["k_pool"], s["v_pool"], case["page"], s["table"], s["q_start"], s["length"], s["out"],
                                 s["ws"], max_new=max(s["new"]), window=case["window"], cap=case["cap"], slopes=s["slopes"])
        return s["out"]
    if op == "beam":
        if not own:
            return _beam(s)
        _nt().nt_beam_select(s["logits"], s["scores"], case["W"], s["parent"], s["token"], s["score"], s["ws"], done=s["done"],
                             done_out=s["done_out"], eos=s["eos"], lengths=s["lengths"], alpha=case["alpha"])
        return s["parent"], s["token"], s["score"], s["done_out"]
    if not own:
        return _pages(s) if op == "pages" else _compact(s)
    nt, page, Hkv, D = _nt(), case["page"], case["Hkv"], case["D"]
    t_stride = s["cache"].shape[3]
    s["refs"].copy_(s["refs_before"])
    if op == "pages":
        nt.nt_page_fork(s["table"], s["length"], s["parent"], s["refs"], page, s["table_out"], s["length_out"])
        nt.nt_page_extend(s["table_out"], s["length_out"], s["refs"], s["q_start"], page, s["rows"], s["pos"], s["pairs"])
        nt.nt_page_copy(s["k_caches"], s["v_caches"], Hkv, D, t_stride, page, s["pairs"])
        return s["refs"], s["table_out"], s["length_out"], s["rows"], s["pos"], s["pairs"], s["cache"]
    s["table"].copy_(s["table_before"])
    nt.nt_page_compact(s["refs"], s["table"], s["length"], page, s["pairs"], s["n_used"], s["ws"])
    nt.nt_page_copy(s["k_caches"], s["v_caches"], Hkv, D, t_stride, page, s["pairs"])
    return s["refs"], s["table"], s["pairs"], s["n_used"], s["cache"]


# ---- cost and definition -------------------------------------------------------------------
def work(case):
    if case["op"] == "attend":
        Hq, Hkv, D, w = case["Hq"], case["Hkv"], case["D"], case["window"]
        size = 4 if case["dtype"] == "f32" else 2
        rows = tokens = pairs = 0
        for n, before in _sequences(case):
            rows += min(n + before, n + w - 1) if w else n + before
            tokens += n
            at = np.arange(before + 1, before + n + 1)
            pairs += int((np.minimum(at, w) if w else at).sum())
        return dict(bytes=2 * 2 * Hkv * rows * D + 2 * size * tokens * Hq * D + 4 * rows // case["page"], flops=4 * pairs * Hq * D)
    if case["op"] == "beam":
        n, k = case["groups"] * case["W"], case["groups"] * case["K"]
        return dict(bytes=4 * n * case["V"] + 12 * n + 16 * k, flops=4 * n * case["V"])
    row = 2 * 2 * case["L"] * case["Hkv"] * case["D"]  # keys and values of a row in every layer
    if case["op"] == "pages":
        S = case["groups"] * case["W"]
        entries = S * ((case["prompt"] + case["since"]) // case["page"] + 1)
        w = np.arange(case["W"] + 1) / case["W"]  # beams that go on, of a request, as `prepare` draws them
        copies = int(S - case["groups"] * (1 - (1 - np.diff(w ** 0.5)) ** case["W"]).sum())
        return dict(bytes=2 * copies * case["page"] * row + 4 * 3 * entries, flops=4 * entries)
    moves = int(case["pages"] * case["used"] * (1 - case["used"]))
    return dict(bytes=2 * moves * case["page"] * row + 4 * 4 * case["pages"], flops=4 * case["pages"])


def _exact_attend(s):
    case = s["case"]
    Hq, D, page = case["Hq"], case["D"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    table, first = s["table"].tolist(), s["q_start"].tolist()
    for i, seen in enumerate(s["length"].tolist()):
        rows = torch.tensor([table[i][t // page] * page + t % page for t in range(seen)], device=DEV)
        n = first[i + 1] - first[i]
        position = torch.arange(seen, device=DEV, dtype=torch.float64)
        for lo in range(0, n, 1024):
            mine = slice(first[i] + lo, first[i] + min(n, lo + 1024))
            me = position[seen - n + lo:][:mine.stop - mine.start, None]
            hidden = position > me
            if case["window"]:
                hidden = hidden | (position <= me - case["window"])
            for h in range(Hq):
                g = h * case["Hkv"] // Hq
                score = s["q"][mine, h].double() @ s["k_pool"][g, rows].double().T / D ** 0.5
                if case["cap"]:
                    score = (score / case["cap"]).tanh() * case["cap"]
                if s["slopes"] is not None:
                    score = score + s["slopes"][h].double() * (position - me)
                score[hidden] = -math.inf
                out[mine, h] = score.softmax(-1) @ s["v_pool"][g, rows].double()
    return out


def _exact_beam(s):
    case = s["case"]
    G, W, K = case["groups"], case["W"], case["K"]
    scores = np.full((G, K), -np.inf)
    done, length, before = (s[k].cpu().numpy() for k in ("done", "lengths", "scores"))
    for i in range(G):
        found = []
        for b in range(i * W, (i + 1) * W):
            if done[b]:
                found.append((float(before[b]) / float(length[b]) ** case["alpha"], float(before[b])))
                continue
            p = torch.log_softmax(s["logits"][b].double(), 0)
            best = p.topk(min(K, len(p))).values.cpu().numpy() + float(before[b])
            found += [(x / (length[b] + 1.0) ** case["alpha"], x) for x in best]
        found.sort(key=lambda pair: -pair[0])
        scores[i, :min(K, len(found))] = [x for _, x in found[:K]]
    return None, None, torch.from_numpy(scores.reshape(-1)), None


def _exact_pages(s):
    """Page by page, as a list of sequences would be kept on the host."""
    page, new = s["case"]["page"], s["case"]["new"]
    table, length, parent, refs = (s[k].cpu().numpy() for k in ("table", "length", "parent", "refs_before"))
    refs = refs.astype(np.int64)
    pool = s["cache"].double()
    held = [list(table[p, :-(-length[p] // page)]) if p >= 0 else [] for p in parent]
    refs[:] = 0
    for pages in held:
        for p in pages:
            refs[p] += 1
    free = [p for p in range(len(refs)) if refs[p] == 0][::-1]
    for pages, up in zip(held, parent):
        n = int(length[up]) if up >= 0 else 0
        if n % page and refs[pages[-1]] > 1:
            refs[pages[-1]] -= 1
            to = free.pop()
            pool[:, :, :, to * page:(to + 1) * page] = s["cache"][:, :, :, pages[-1] * page:(pages[-1] + 1) * page].double()
            pages[-1] = to
        pages += [free.pop() for _ in range(-(-(n + new) // page) - len(pages))]
    return None, None, None, None, None, None, pool


def _exact_compact(s):
    page = s["case"]["page"]
    used = s["refs_before"].cpu().numpy() > 0
    count = int(used.sum())
    pool = s["cache"].double()
    for to, at in zip(np.flatnonzero(~used[:count]), count + np.flatnonzero(used[count:])):
        pool[:, :, :, to * page:(to + 1) * page] = s["cache"][:, :, :, at * page:(at + 1) * page]
    return None, None, None, None, pool


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "beam": _exact_beam, "pages": _exact_pages, "compact": _exact_compact}[case["op"]](s)
