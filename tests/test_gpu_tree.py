"""The tree-verify operators on the GPU against plain 64-bit implementations. Tolerances count
roundings: fp32 2^-24, bf16 2^-8 of the value each; sums of n terms are allowed sqrt(n) of them."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests import _tree
from tests._gpu import DEV, dev, host

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, tol, what=""):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err)}, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]}")


# ---- head norms, rotation, append -----------------------------------------------------------
def run_append(B, Hq, Hkv, D, rd, layout, dtype, norm=True, fused=False, pos=None, pos0=11, rows=None, row0=3, ts=None,
               amplitude=1.0, base=1e4, alias=False, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[dtype]
    qkv = (torch.randn(B, Hq + 2 * Hkv, D, generator=g, device=DEV) * 2).to(t)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qg, kg = (1 + 0.3 * torch.randn(D, generator=g, device=DEV) if norm else None for _ in range(2))
    f = base ** (-np.arange(rd // 2) * 2.0 / max(rd, 1))
    ts = ts or row0 + B + 2
    kc, vc = (torch.full((Hkv, ts, D), -7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    qin = f64(q)
    out = q if alias else torch.full((B, Hq, D), float("nan"), dtype=t, device=DEV)
    n_bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    nt.nt_qk_norm_rope_append(q, k, v, qg, kg, 1e-6, dev(f) if rd else None, layout, amplitude, out, kc, vc,
                              pos=None if pos is None else dev(pos.astype(np.int32)), pos0=pos0,
                              rows=None if rows is None else dev(rows.astype(np.int32)), row0=row0, n_bad=n_bad)
    p = pos if pos is not None else pos0 + np.arange(B)
    r = rows if rows is not None else row0 + np.arange(B)
    gam = lambda x: None if x is None else f64(x)  # noqa: E731
    wq = _tree.rotate(qin, gam(qg), 1e-6, f, layout, amplitude, p)
    wk = _tree.rotate(f64(k), gam(kg), 1e-6, f, layout, amplitude, p)

    # the norm: sqrt(D) roundings of the sum halved by the root, 4 for mean, root, quotient, product
    # and gain; sine and cosine 2 ulp and half an angle ulp of up to pi (3); three more products and
    # a sum: 16 + sqrt(D) / 2 roundings of a pair's size
    def bound(w):
        size = np.abs(w).max(-1, keepdims=True) * 1.5
        return (16 + D ** 0.5 / 2) * U32 * size

    within(f64(out), wq, bound(wq) + (U16 * np.abs(wq) if dtype == "bf16" else 0), "q")
    kcn, vcn = f64(kc), f64(vc)
    ok = [(b, r[b]) for b in range(B) if 0 <= r[b] < ts]
    bs, rs = [b for b, _ in ok], [row for _, row in ok]
    within(kcn[:, rs], wk[bs].transpose(1, 0, 2), (bound(wk) + U16 * np.abs(wk))[bs].transpose(1, 0, 2), "k")
    assert np.array_equal(vcn[:, rs], f64(v.to(torch.bfloat16))[bs].transpose(1, 0, 2))
    untouched = np.ones(ts, bool)
    untouched[rs] = False
    assert (kcn[:, untouched] == -7.0).all() and (vcn[:, untouched] == -7.0).all()
    assert int(n_bad) == B - len(ok)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("B,Hq,Hkv,D,rd", [(1, 32, 8, 128, 128), (5, 3, 3, 64, 64), (7, 14, 2, 128, 64), (3, 4, 1, 256, 64),
                                           (2, 6, 2, 96, 24), (33, 8, 8, 8, 8), (4, 5, 5, 40, 0), (64, 32, 4, 64, 16),
                                           (2, 1, 1, 256, 256), (1, 70, 10, 128, 120)])
def test_append(B, Hq, Hkv, D, rd, layout, dtype):
    run_append(B, Hq, Hkv, D, rd, layout, dtype, fused=B % 2 == 0, norm=B != 5)


@pytest.mark.parametrize("pos0", [0, 1, 4095, 131071, 1 << 20, (1 << 31) - 4])
def test_append_far_positions(pos0):
    # the 64-bit reference forms the angle in double: its own error is pos * 2^-53 * 2 radians
    run_append(3, 4, 2, 128, 128, 0, "f32", pos0=pos0)
    run_append(3, 4, 2, 64, 32, 1, "f32", pos0=pos0, amplitude=1.14, base=1e6)


def test_append_negative_and_device_positions_and_rows():
    rs = np.random.RandomState(1)
    run_append(9, 4, 2, 64, 64, 1, "f32", pos=rs.randint(-100000, 100000, 9), rows=rs.permutation(20)[:9], ts=20)
    run_append(6, 4, 2, 128, 128, 0, "bf16", pos=np.full(6, 77), rows=np.array([5, -1, 19, 20, 2 ** 31 - 1, 0]), ts=20)


def test_append_in_place_and_many_tokens():
    run_append(17, 8, 2, 128, 128, 0, "f32", alias=True)
    run_append(2049, 8, 2, 128, 128, 0, "bf16", fused=True)
    run_append(1500, 30, 3, 64, 64, 1, "f32", fused=True)


def test_append_and_attention_beyond_32_bit_offsets():
    ts, D = (1 << 31) // 128 // 2 + 100, 128
    kc, vc = (torch.zeros(3, ts, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))  # > 2^31 elements
    assert kc.numel() > 2 ** 31
    q, k, v = torch.randn(2, 3, D, device=DEV), torch.randn(2, 3, D, device=DEV), torch.randn(2, 3, D, device=DEV)
    out = torch.empty_like(q)
    nt.nt_qk_norm_rope_append(q, k, v, None, None, 0.0, None, 0, 1.0, out, kc, vc, row0=ts - 2)
    assert torch.equal(out, q)
    assert torch.equal(kc[:, ts - 2:], k.transpose(0, 1).bfloat16()) and torch.equal(vc[:, ts - 2:], v.transpose(0, 1).bfloat16())
    mask = torch.from_numpy(_tree.pack(np.eye(2, dtype=bool))).to(DEV)
    ws = torch.zeros(nt.nt_tree_attention_workspace_size(2, 3, 3, D, 0), dtype=torch.uint8, device=DEV)
    nt.nt_tree_attention(q, kc, vc, 0, ts - 2, mask, out, ws)  # each node sees its own row alone
    assert torch.equal(out, v.bfloat16().float())


@pytest.mark.parametrize("scaling", [0, 1, 2])
def test_frequencies(scaling):
    f = torch.empty(48, dtype=torch.float64, device=DEV)
    nt.nt_rope_frequencies(96, 5e5, f, scaling, factor=8.0, trained_len=8192, slow=1.0, fast=4.0)
    want = 5e5 ** (-np.arange(48) / 48.0)
    if scaling == 1:
        want = want / 8
    if scaling == 2:
        w = np.clip((8192 * want / (2 * np.pi) - 1) / 3, 0, 1)
        assert (w == 0).any() and (w == 1).any() and ((w > 0) & (w < 1)).any()
        want = want * (w + (1 - w) / 8)
    within(f64(f), want, 2.0 ** -48 * want)


# ---- tree layout, acceptance, commit ---------------------------------------------------------
@pytest.mark.parametrize("shape", ["chain", "star", "tree", "forest"])
@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 64, 200, 256])
def test_layout(B, shape):
    p = _tree.parents(np.random.RandomState(B), B, shape)
    words = (B + 31) // 32 + (B % 2)
    mask = torch.full((B, words), -1, dtype=torch.int32, device=DEV)
    pos = torch.empty(B, dtype=torch.int32, device=DEV)
    nt.nt_tree_layout(dev(p), mask, pos, 1000)
    seen = _tree.ancestors(p)
    assert np.array_equal(host(mask), _tree.pack(seen, words))
    assert np.array_equal(host(pos), 999 + seen.sum(1))


def test_layout_bad_parents_are_roots():
    p = np.array([-1, 1, 7, 2, 3, -9], dtype=np.int32)
    n_bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    mask = torch.empty(6, 1, dtype=torch.int32, device=DEV)
    nt.nt_tree_layout(dev(p), mask, n_bad=n_bad)
    want = np.eye(6, dtype=bool)
    want[3, 2] = want[4, 2] = want[4, 3] = True
    assert np.array_equal(host(mask), _tree.pack(want)) and int(n_bad) == 2


@pytest.mark.parametrize("shape", ["chain", "star", "tree", "forest"])
@pytest.mark.parametrize("B", [1, 2, 9, 64, 255, 256])
@pytest.mark.parametrize("vocab", [2, 50])
def test_accept(B, shape, vocab):
    rs = np.random.RandomState(B + vocab)
    for _ in range(4):
        p = _tree.parents(rs, B, shape)
        token, am = (rs.randint(0, vocab, B).astype(np.int32) for _ in range(2))
        if shape == "chain":  # agree for a while
            n = B // 2
            am[:n] = token[1:n + 1]
        emit, path = (torch.empty(B, dtype=torch.int32, device=DEV) for _ in range(2))
        n = torch.empty(1, dtype=torch.int32, device=DEV)
        nt.nt_tree_accept(dev(p), dev(token), dev(am), emit, path, n)
        wp, we = _tree.accept(p, token, am)
        fill = [-1] * (B - len(wp))
        assert int(n) == len(wp) and host(path).tolist() == wp + fill and host(emit).tolist() == we + fill


def test_accept_of_a_chain_is_verify_accept():
    rs = np.random.RandomState(3)
    for B in (1, 4, 16):
        draft, am = rs.randint(0, 2, B - 1).astype(np.int32), rs.randint(0, 2, B).astype(np.int32)
        emit, path, e2 = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
        n, n2 = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
        token = np.concatenate([[99], draft]).astype(np.int32)
        nt.nt_tree_accept(dev(np.arange(-1, B - 1, dtype=np.int32)), dev(token), dev(am), emit, path, n)
        nt.nt_verify_accept(dev(draft) if B > 1 else None, dev(am), B, e2, n2)
        assert int(n) == int(n2) and torch.equal(emit[:int(n)], e2[:int(n)])


@pytest.mark.parametrize("L,Hkv,D", [(1, 1, 8), (3, 2, 64), (2, 5, 128), (130, 1, 16), (1, 3, 256)])
@pytest.mark.parametrize("src,dst", [(10, 10), (10, 7), (40, 3), (11, 10)])
def test_commit(L, Hkv, D, src, dst):
    rs = np.random.RandomState(src)
    B, ts = 20, 64
    for n in (0, 1, 4, 5, 20):
        path = np.full(B, -1, dtype=np.int32)
        path[:n] = np.sort(rs.permutation(B)[:n])
        k, v = (torch.randn(L, Hkv, ts, D, device=DEV).bfloat16() for _ in range(2))
        want = []
        for c in (k, v):
            w = c.clone()
            w[:, :, dst:dst + n] = c[:, :, torch.from_numpy(src + path[:n].astype(np.int64)).to(DEV)]
            want.append(w)
        nt.nt_tree_commit(nt.pointer_array(list(k)), nt.pointer_array(list(v)), Hkv, D, ts, dev(path),
                          torch.tensor([n], dtype=torch.int32, device=DEV), src, dst)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_commit_ignores_entries_out_of_range():
    k = torch.randn(1, 1, 32, 8, device=DEV).bfloat16()
    v, k0 = k.clone(), k.clone()
    path = np.array([0, 4, -1, 1, 2 ** 30], dtype=np.int32)  # entries 2..4 are below their place or past B
    nt.nt_tree_commit(nt.pointer_array([k[0]]), nt.pointer_array([v[0]]), 1, 8, 32, dev(path),
                      torch.tensor([1000], dtype=torch.int32, device=DEV), 10, 3)
    k0[:, :, 3], k0[:, :, 4] = k0[:, :, 10].clone(), k0[:, :, 14].clone()
    assert torch.equal(k, k0) and torch.equal(v, k0)


# ---- logits ----------------------------------------------------------------------------------
def run_adjust(B, V, paths, mask, bias, want_out=True, want_arg=True, rep=1.25, freq=0.375, pres=0.5, seed=0, strided=False,
               inplace=False):
    rs = np.random.RandomState(seed)
    x = (rs.randn(B, V) * 3).astype(np.float32)
    shared = rs.binomial(3, 0.05, (B if strided else 1, V)).astype(np.int32)
    counts = np.broadcast_to(shared, (B, V)).copy()
    tm = tok = None
    if paths:
        seen = _tree.ancestors(_tree.parents(rs, B))
        tok = rs.randint(0, V, B).astype(np.int32)
        tok[rs.rand(B) < 0.3] = V - 1
        tok[rs.rand(B) < 0.1] = -1  # outside the vocabulary: counts nowhere
        for b in range(B):
            for j in np.flatnonzero(seen[b]):
                if 0 <= tok[j] < V:
                    counts[b, tok[j]] += 1
        tm = dev(_tree.pack(seen))
    bi = None if not bias else (rs.randn(B if strided else 1, V) * (rs.rand(1, V) < 0.1)).astype(np.float32)
    al = None
    if mask:
        al = rs.rand(1 if mask == "shared" else B, V) < 0.3
        if mask == "empty":
            al[:] = False
    ws = torch.zeros(nt.nt_logits_adjust_workspace_size(V, B), dtype=torch.uint8, device=DEV)
    dx = dev(x)
    out = (dx if inplace else torch.full((B, V), 5.0, device=DEV)) if want_out else None
    am = torch.full((B,), -9, dtype=torch.int32, device=DEV) if want_arg else None
    for _ in range(1 if inplace else 2):  # the workspace is left zero
        nt.nt_logits_adjust(dx, counts=dev(shared), tree_mask=tm, tokens=None if tok is None else dev(tok), repetition=rep,
                            frequency=freq, presence=pres, bias=None if bi is None else dev(bi),
                            allowed=None if al is None else dev(_tree.pack(al)), out=out, argmax=am, ws=ws)
        assert not ws.any()
    w32 = _tree.adjust(x, counts, rep, freq, pres, bi, al, np.float32)
    w64 = _tree.adjust(x, counts, rep, freq, pres, bi, al)
    if want_out:
        # each of the five steps rounds once, relative to the largest value it meets
        size = np.abs(x) * max(rep, 1 / rep) + abs(freq) * counts + abs(pres) + (0 if bi is None else np.abs(bi))
        y = host(out)
        fin = np.isfinite(w64)
        assert np.array_equal(np.isneginf(y), ~fin)
        within(np.where(fin, y, 0), np.where(fin, w64, 0), 5 * U32 * size, "logits")
        assert np.array_equal(y, w32)  # the steps are the header's, rounded one by one
    if want_arg:
        assert np.array_equal(host(am), _tree.choice(w32))


@pytest.mark.parametrize("B,V", [(1, 1), (1, 31), (2, 33), (3, 1023), (5, 1024), (4, 4100), (64, 5000), (2, 151936), (256, 1000),
                                 (7, 32003)])
@pytest.mark.parametrize("paths,mask,bias", [(True, "row", True), (False, "shared", False), (True, None, True), (False, "empty", False)])
def test_adjust(B, V, paths, mask, bias):
    run_adjust(B, V, paths, mask, bias)


def test_adjust_variants():
    run_adjust(5, 2000, True, "row", True, want_out=False)
    run_adjust(5, 2000, True, "row", True, want_arg=False)
    run_adjust(5, 2000, True, "row", True, strided=True)
    run_adjust(5, 2001, True, "row", True, strided=True)
    run_adjust(5, 2004, True, "row", True, inplace=True)
    run_adjust(5, 2001, False, None, True, inplace=True)
    run_adjust(300, 77, False, "row", False)
    run_adjust(6, 3000, True, "row", False, rep=0.5, freq=-1.0, pres=-0.25)


@pytest.mark.parametrize("V", [1000, 1001, 5000])
def test_adjust_ties_nans_and_infinities(V):
    x = np.full((7, V), -1.0, dtype=np.float32)
    x[0, [V - 1, 500, 999]] = 2.0          # ties: the lowest index
    x[1] = -np.inf                          # nothing above -inf
    x[2, 10], x[2, 20] = np.nan, 3.0        # NaN is never chosen
    x[3, 700] = np.inf
    x[4] = np.float32(-0.0)
    x[4, 900] = 0.0                         # +0 and -0 are equal
    x[5] = np.nan
    x[6, 5] = 9.0                           # not allowed
    al = np.ones((7, V), dtype=bool)
    al[6, 5] = False
    am = torch.empty(7, dtype=torch.int32, device=DEV)
    out = torch.empty(7, V, device=DEV)
    ws = torch.zeros(nt.nt_logits_adjust_workspace_size(V, 7), dtype=torch.uint8, device=DEV)
    nt.nt_logits_adjust(dev(x), allowed=dev(_tree.pack(al)), out=out, argmax=am, ws=ws)
    assert host(am).tolist() == [500, -1, 20, 700, 0, -1, 0]
    y = host(out)
    assert np.array_equal(y[:6], x[:6], equal_nan=True) and y[6, 5] == -np.inf


@pytest.mark.parametrize("V", [6144, 6145])
@pytest.mark.parametrize("every", [1, 2, 3, 4, 5, 40])
def test_adjust_however_many_tokens_are_used(V, every):
    """From all tokens to a few: the kernel lists a few used tokens and works on all of them otherwise."""
    rs = np.random.RandomState(every)
    B = 9
    x = (rs.randn(B, V) * 4).astype(np.float32)
    counts = np.where(np.arange(V) % every == 0, 1 + rs.randint(0, 3, V), 0).astype(np.int32)
    sees = _tree.ancestors(_tree.parents(rs, B))
    tokens = rs.randint(0, V, B).astype(np.int32)
    tokens[3:6] = tokens[0]  # the same token on several nodes, some of a path
    full = np.stack([counts + np.bincount(tokens[s], minlength=V) for s in sees]).astype(np.int32)
    want = _tree.adjust(x, full, 1.3, 0.25, -0.5, None, None, np.float32)
    out = torch.empty(B, V, device=DEV)
    arg = torch.empty(B, dtype=torch.int32, device=DEV)
    ws = torch.zeros(nt.nt_logits_adjust_workspace_size(V, B), dtype=torch.uint8, device=DEV)
    nt.nt_logits_adjust(dev(x), counts=dev(counts), tree_mask=dev(_tree.pack(sees)), tokens=dev(tokens), repetition=1.3,
                        frequency=0.25, presence=-0.5, out=out, argmax=arg, ws=ws)
    assert np.array_equal(host(out), want)
    assert np.array_equal(host(arg), _tree.choice(want))


@pytest.mark.parametrize("rep", [1.1, 1.0, 1.25, 3.0, 0.7, 1.9999999, 1e-5, 7e4, 1e-30, 1e30])
def test_adjust_quotients_are_rounded(rep):
    """Every significand of one binade, and values of any size, divided as IEEE division does."""
    sig = (np.arange(1 << 23, dtype=np.uint32) | np.uint32(127 << 23)).view(np.float32)
    rs = np.random.RandomState(1)
    odd = rs.randint(0, 0x7f800000, 1 << 16).astype(np.uint32).view(np.float32)
    x = np.concatenate([sig, odd, -odd, np.float32([0.0, -0.0, np.inf, -np.inf, 1e-45])])
    out = torch.empty(1, x.size, device=DEV)
    nt.nt_logits_adjust(dev(x[None]), counts=torch.ones(x.size, dtype=torch.int32, device=DEV), repetition=rep, out=out)
    with np.errstate(over="ignore", under="ignore"):
        r = np.float32(rep)
        want = np.where(x > 0, x / r, x * r)
    assert np.array_equal(host(out)[0], want)


def test_token_counts():
    rs = np.random.RandomState(0)
    for n in (0, 1, 255, 70000):
        tok = rs.randint(-2, 52, n).astype(np.int32)
        counts, n_bad = torch.ones(50, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        nt.nt_token_counts(dev(tok), counts, n_bad=n_bad)
        ok = (tok >= 0) & (tok < 50)
        assert np.array_equal(host(counts), 1 + np.bincount(tok[ok], minlength=50)) and int(n_bad) == n - ok.sum()
    tok, idx = dev(np.array([3, 4, 5, 6], dtype=np.int32)), dev(np.array([0, 2, 2, -1], dtype=np.int32))
    for n, want in ((3, {3: 1, 5: 2}), (9, {3: 1, 5: 2}), (0, {}), (-4, {})):
        counts = torch.zeros(8, dtype=torch.int32, device=DEV)
        nt.nt_token_counts(tok, counts, index=idx, n=torch.tensor([n], dtype=torch.int32, device=DEV))
        assert host(counts).tolist() == [want.get(i, 0) for i in range(8)]


# ---- attention ---------------------------------------------------------------------------------
def attn_inputs(B, Hq, Hkv, D, prefix, gap, dtype, seed=0, scale=1.5, tail=3):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ts = prefix + gap + B + tail
    q = (torch.randn(B, Hq, D, generator=g, device=DEV) * scale).to(TYPES[dtype])
    k, v = (torch.randn(Hkv, ts, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    return q, k, v


def run_attend(q, k, v, prefix, row0, sees, runs=1, words=None):
    B, Hq, D = q.shape
    ws = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hq, k.shape[0], D, prefix), dtype=torch.uint8, device=DEV)
    mask = dev(_tree.pack(sees, words))
    outs = []
    for _ in range(runs):
        out = torch.full_like(q, float("nan"))
        nt.nt_tree_attention(q, k, v, prefix, row0, mask, out, ws)
        torch.cuda.synchronize()
        assert nt.nt_workspace_status(ws) == nt.NT_OK
        outs.append(out)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])  # the same inputs, the same bits
    return outs[0]


def attn_bound(q, k, v, prefix, sees, dtype, want):
    """A score's error: sqrt(D) roundings of |q| |k| / sqrt(D) (half a step or a truncation: 2 U32 each);
    a weight's is that, twice (its own and the sum's); the weighted sum adds sqrt(keys) roundings
    and a few for exponentials, joins and the quotient. All relative to the largest value."""
    D = q.shape[-1]
    qn, kn = float(q.double().norm(dim=-1).max()), float(k.double().nan_to_num(0, 0, 0).norm(dim=-1).max())
    vm = float(v.double().nan_to_num(0, 0, 0).abs().max())
    keys = prefix + q.shape[0]
    tol = vm * 2 * U32 * (2 * D ** 0.5 * qn * kn / D ** 0.5 + keys ** 0.5 + 16)
    return tol + (U16 * np.abs(want) if dtype == "bf16" else 0)


def check_attend(B, Hq, Hkv, D, prefix, gap, dtype, shape="tree", seed=0, runs=1):
    q, k, v = attn_inputs(B, Hq, Hkv, D, prefix, gap, dtype, seed)
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(seed), B, shape))
    out = run_attend(q, k, v, prefix, prefix + gap, sees, runs)
    want = _tree.attend(f64(q), f64(k), f64(v), prefix, prefix + gap, sees)
    within(f64(out), want, attn_bound(q, k, v, prefix, sees, dtype, want), "out")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,prefix,gap", [
    (1, 1, 1, 0, 0), (1, 4, 1, 1, 0), (1, 32, 8, 63, 0), (2, 8, 2, 64, 5), (3, 8, 8, 65, 0), (8, 32, 8, 127, 1), (9, 12, 4, 128, 0),
    (16, 8, 1, 129, 0), (25, 32, 8, 500, 0), (33, 4, 1, 31, 40), (64, 8, 2, 1000, 0), (65, 10, 2, 191, 0), (100, 7, 1, 257, 3),
    (128, 4, 4, 0, 0), (200, 8, 1, 66, 0), (256, 4, 2, 320, 0)])
def test_attention(B, Hq, Hkv, prefix, gap, D, dtype):
    check_attend(B, Hq, Hkv, D, prefix, gap, dtype, seed=B + prefix)


@pytest.mark.parametrize("shape", ["chain", "star", "forest"])
def test_attention_shapes(shape):
    check_attend(40, 8, 2, 128, 100, 0, "f32", shape)
    check_attend(130, 4, 2, 64, 70, 9, "bf16", shape)


@pytest.mark.parametrize("B,prefix", [(1, 8191), (4, 20000), (40, 9001)])
def test_attention_long(B, prefix):
    check_attend(B, 8, 2, 128, prefix, 0, "f32", runs=2)


def test_attention_many_heads():
    check_attend(2, 200, 200, 64, 130, 0, "f32")   # more heads than SMs
    check_attend(3, 320, 2, 128, 70, 0, "f32")     # 160 query heads share one


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 8, 8), (2, 16, 4), (3, 20, 2), (7, 32, 8), (32, 3, 3), (9, 32, 8), (32, 14, 2), (25, 32, 8)])
def test_attention_few_rows_of_every_length(B, Hq, Hkv, dtype, D):
    """Up to 32 rows per key-value head, and more of up to 32 nodes: unsplit, in clusters, in splits; odd numbers of tiles."""
    for prefix in (0, 1, 62, 64, 65, 300, 383, 447, 448, 449, 511, 900, 1500, 2303, 5900, 6079, 6080, 6144, 6200, 9000):
        q, k, v = attn_inputs(B, Hq, Hkv, D, prefix, 2, dtype, seed=prefix)
        sees = _tree.ancestors(_tree.parents(np.random.RandomState(prefix), B))
        out = f64(run_attend(q, k, v, prefix, prefix + 2, sees, runs=2))
        want = attend_64(q, k, v, prefix, prefix + 2, sees)
        within(out, want, attn_bound(q, k, v, prefix, sees, dtype, want), prefix)


def attend_64(q, k, v, prefix, row0, sees):
    """_tree.attend for many heads at a time."""
    (B, Hq, D), Hkv = q.shape, k.shape[0]
    rows = torch.cat([torch.arange(prefix, device=DEV), torch.arange(row0, row0 + B, device=DEV)])
    seen = torch.cat([torch.ones(B, prefix, dtype=torch.bool, device=DEV), dev(sees)], dim=1)
    qd = q.double().view(B, Hkv, Hq // Hkv, D)
    s = torch.einsum("bhgd,htd->hgbt", qd, k[:, rows].double()) / D ** 0.5
    w = s.masked_fill(~seen, float("-inf")).softmax(-1)
    return f64(torch.einsum("hgbt,htd->bhgd", w, v[:, rows].double()).reshape(B, Hq, D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [2, 12, 30, 40, 70, 133])
@pytest.mark.parametrize("kind", ["random", "rise"])
def test_attention_many_tiles_to_a_block(B, D, kind):
    """A head to a block (more heads than SMs), so that one block walks every tile count about the
    points where the accumulator is taken to registers; also with a maximum that keeps rising."""
    Hkv = 160
    for tiles in (1, 2, 3, 7, 8, 9, 10, 15, 16, 17, 18, 24, 25):
        prefix = max(0, 64 * tiles - 64 * ((B + 63) // 64) - (tiles % 3) * 9)
        q, k, v = attn_inputs(B, Hkv, Hkv, D, prefix, 0, "f32", seed=tiles)
        if kind == "rise":
            ramp = torch.linspace(0, 10, k.shape[1], device=DEV)
            k = (k * 0.1 + ramp[None, :, None] * q.mean(0)[:, None] / q.mean(0).norm(dim=-1)[:, None, None]).bfloat16()
        sees = _tree.ancestors(_tree.parents(np.random.RandomState(tiles), B))
        out = run_attend(q, k, v, prefix, prefix, sees, runs=2)
        want = attend_64(q, k, v, prefix, prefix, sees)
        within(f64(out), want, attn_bound(q, k, v, prefix, sees, "f32", want), (kind, tiles))


@pytest.mark.parametrize("B,Hq,Hkv,prefix,dtype,D", [
    (40, 160, 160, 2000, "f32", 64), (40, 160, 160, 2100, "bf16", 128), (200, 64, 8, 4000, "f32", 128), (200, 64, 8, 4011, "bf16", 64),
    (255, 32, 4, 12000, "f32", 64), (70, 300, 300, 1500, "f32", 128)])
@pytest.mark.parametrize("kind", ["random", "rise", "non-finite"])
def test_attention_equal_shares(B, Hq, Hkv, prefix, dtype, D, kind):
    """Numbers of row tiles that do not fill the GPU evenly: blocks begin and end within a row tile."""
    q, k, v = attn_inputs(B, Hq, Hkv, D, prefix, 1, dtype, seed=B)
    if kind == "rise":
        ramp = torch.linspace(0, 10, k.shape[1], device=DEV)
        u = q.float().view(B, Hkv, -1, D).mean((0, 2))
        k = (k * 0.1 + ramp[None, :, None] * (u / u.norm(dim=-1, keepdim=True))[:, None]).bfloat16()
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(B), B))
    bad = B - 1  # seen by itself alone
    if kind == "non-finite":
        v[:, prefix + 1 + bad] = float("inf")
        k[:, prefix] = v[:, prefix] = float("nan")  # between the sequence and the tree
    out = f64(run_attend(q, k, v, prefix, prefix + 1, sees, runs=2))
    want = attend_64(q, k, v.nan_to_num(0, 0, 0), prefix, prefix + 1, sees)
    if kind == "non-finite":
        assert np.isposinf(out[bad]).all()
        out, want, sees = out[:bad], want[:bad], sees[:bad]
    within(out, want, attn_bound(q, k, v, prefix, sees, dtype, want), kind)


def test_attention_chain_matches_the_chain_call():
    q, k, v = attn_inputs(6, 32, 8, 128, 700, 0, "f32", tail=0)
    sees = np.tril(np.ones((6, 6), bool))
    got = run_attend(q, k, v, 700, 700, sees)
    out = torch.empty_like(q)
    ws = torch.zeros(nt.nt_attention_workspace_size(6, 32, 8, 706), dtype=torch.uint8, device=DEV)
    nt.nt_attention_decode(q, k.view(torch.int16), v.view(torch.int16), 6, 32, 8, 128, 706, k.shape[1], out, ws)
    within(f64(got), f64(out), 2 * attn_bound(q, k, v, 700, sees, "f32", f64(out)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [5, 70])
def test_attention_empty_rows(B, D, dtype):
    q, k, v = attn_inputs(B, 8, 2, D, 0, 0, dtype)
    sees = np.random.RandomState(0).rand(B, B) < 0.2  # any bits, not only a tree's
    sees[[0, B // 2]] = False
    out = run_attend(q, k, v, 0, 0, sees)
    want = _tree.attend(f64(q), f64(k), f64(v), 0, 0, sees)
    assert (out[0] == 0).all() and (out[B // 2] == 0).all()
    within(f64(out), want, attn_bound(q, k, v, 0, sees, dtype, want))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("B,prefix,gap", [(6, 100, 7), (70, 64, 1), (1, 0, 3), (129, 10, 70)])
def test_attention_what_is_masked_has_no_part(B, prefix, gap, bad):
    for D, dtype in ((128, "f32"), (64, "bf16")):
        q, k, v = attn_inputs(B, 8, 2, D, prefix, gap, dtype, tail=40)
        sees = _tree.ancestors(_tree.parents(np.random.RandomState(1), B))
        lone = B - 1  # a node that no one sees
        sees[:, lone] = False
        row0 = prefix + gap
        want = _tree.attend(f64(q), f64(k), f64(v), prefix, row0, sees)
        for c in (k, v):
            c[:, prefix:row0] = bad          # between the sequence and the tree
            c[:, row0 + B:] = bad            # past the tree
            c[:, row0 + lone] = bad
        out = run_attend(q, k, v, prefix, row0, sees)
        within(f64(out), want, attn_bound(q, k, v, prefix, sees, dtype, want))


def test_attention_non_finite_values_reach_only_those_that_see_them():
    B, prefix = 40, 70
    for D, dtype in ((128, "f32"), (64, "bf16")):
        q, k, v = attn_inputs(B, 4, 2, D, prefix, 0, dtype)
        sees = _tree.ancestors(_tree.parents(np.random.RandomState(2), B))
        clean = _tree.attend(f64(q), f64(k), f64(v), prefix, prefix, sees)
        tol = attn_bound(q, k, v, prefix, sees, dtype, clean)
        v[:, prefix + 7, 3], v[:, prefix + 9, 5] = float("inf"), float("nan")
        out = f64(run_attend(q, k, v, prefix, prefix, sees))
        fine = np.ones((B, D), bool)
        fine[sees[:, 7], 3] = fine[sees[:, 9], 5] = False
        fine = np.broadcast_to(fine[:, None], out.shape)
        within(np.where(fine, out, 0), np.where(fine, clean, 0), tol)
        assert not np.isfinite(out[sees[:, 7]][:, :, 3]).any() and np.isnan(out[sees[:, 9]][:, :, 5]).all()
        k[:, prefix + 11] = float("nan")  # a key: every weight of those that see it
        out = f64(run_attend(q, k, v, prefix, prefix, sees))
        assert np.isnan(out[sees[:, 11]]).all()
        rest = fine & ~sees[:, 11][:, None, None]
        within(np.where(rest, out, 0), np.where(rest, clean, 0), tol)


def test_attention_large_and_flat_scores():
    """One key far above the others; all keys alike; a maximum that rises through the sequence."""
    for D in (64, 128):
        q, k, v = attn_inputs(20, 8, 2, D, 900, 0, "f32", scale=1.0)
        sees = _tree.ancestors(_tree.parents(np.random.RandomState(3), 20))
        for kind in ("peak", "flat", "rise", "fall"):
            kk = k.clone()
            if kind == "peak":
                kk[:, 500] = (q[0, 0] * 8).bfloat16()
            if kind == "flat":
                kk[:] = kk[:, :1]
            if kind in ("rise", "fall"):
                ramp = torch.linspace(0, 12, kk.shape[1], device=DEV)
                kk = (kk * 0.1 + (ramp if kind == "rise" else ramp.flip(0))[None, :, None] * q.mean((0, 1)) * 4).bfloat16()
            out = run_attend(q, kk, v, 900, 900, sees)
            want = _tree.attend(f64(q), f64(kk), f64(v), 900, 900, sees)
            within(f64(out), want, attn_bound(q, kk, v, 900, sees, "f32", want), kind)


def test_attention_bits_past_the_tree_do_not_count():
    q, k, v = attn_inputs(5, 8, 2, 128, 40, 0, "f32")
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(4), 5))
    wide = np.ones((5, 96), bool)
    wide[:, :5] = sees
    a = run_attend(q, k, v, 40, 40, sees)
    assert torch.equal(a, run_attend(q, k, v, 40, 40, wide, words=3))


def test_attention_timeout_is_reported_until_cleared():
    q, k, v = attn_inputs(9, 8, 2, 128, 400, 0, "f32")
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(6), 9))
    want = run_attend(q, k, v, 400, 400, sees)
    ws = torch.zeros(nt.nt_tree_attention_workspace_size(9, 8, 2, 128, 400), dtype=torch.uint8, device=DEV)
    mask, out = dev(_tree.pack(sees)), torch.empty_like(q)
    try:
        nt.nt_set_test_fault(5, 20.0)
        nt.nt_tree_attention(q, k, v, 400, 400, mask, out, ws)
        torch.cuda.synchronize()
    finally:
        nt.nt_set_test_fault(0)
    assert nt.nt_workspace_status(ws) == nt.NT_ERR_TIMEOUT
    ws.zero_()
    nt.nt_tree_attention(q, k, v, 400, 400, mask, out, ws)
    torch.cuda.synchronize()
    assert nt.nt_workspace_status(ws) == nt.NT_OK and torch.equal(out, want)


@pytest.mark.parametrize("B,Hq,Hkv,prefix,D,dtype", [
    (3, 8, 2, 400, 128, "f32"), (3, 8, 2, 900, 128, "f32"), (2, 8, 2, 9000, 64, "f32"), (8, 8, 2, 90, 64, "bf16"),
    (40, 160, 160, 2000, 64, "f32")])
def test_attention_timeout_with_few_rows_and_in_shares(B, Hq, Hkv, prefix, D, dtype):
    q, k, v = attn_inputs(B, Hq, Hkv, D, prefix, 0, dtype)
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(6), B))
    want = run_attend(q, k, v, prefix, prefix, sees)
    ws = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hq, Hkv, D, prefix), dtype=torch.uint8, device=DEV)
    mask, out = dev(_tree.pack(sees)), torch.empty_like(q)
    try:
        nt.nt_set_test_fault(5, 20.0)
        nt.nt_tree_attention(q, k, v, prefix, prefix, mask, out, ws)
        torch.cuda.synchronize()
    finally:
        nt.nt_set_test_fault(0)
    assert nt.nt_workspace_status(ws) == nt.NT_ERR_TIMEOUT
    ws.zero_()
    nt.nt_tree_attention(q, k, v, prefix, prefix, mask, out, ws)
    torch.cuda.synchronize()
    assert nt.nt_workspace_status(ws) == nt.NT_OK and torch.equal(out, want)


# ---- streams and graphs --------------------------------------------------------------------------
def test_attention_forms_in_one_graph_and_on_two_streams():
    """Unsplit, in a cluster, in splits, many rows and equal shares: one after the other in a replayed graph, and at once."""
    calls = []
    for B, Hq, Hkv, prefix, D, dtype in [(1, 32, 8, 60, 128, "f32"), (2, 32, 8, 1500, 128, "f32"), (1, 8, 2, 20000, 64, "bf16"),
                                         (25, 32, 8, 2000, 128, "f32"), (40, 160, 160, 2000, 64, "f32"), (7, 32, 8, 900, 64, "bf16")]:
        q, k, v = attn_inputs(B, Hq, Hkv, D, prefix, 0, dtype, seed=prefix)
        sees = _tree.ancestors(_tree.parents(np.random.RandomState(B), B))
        want = run_attend(q, k, v, prefix, prefix, sees)
        ws = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hq, Hkv, D, prefix), dtype=torch.uint8, device=DEV)
        calls.append(((q, k, v, prefix, prefix, dev(_tree.pack(sees))), torch.zeros_like(q), ws, want))
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        for args, out, ws, _ in calls:
            nt.nt_tree_attention(*args, out, ws)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for _, out, ws, want in calls:
            assert nt.nt_workspace_status(ws) == nt.NT_OK and torch.equal(out, want)
            out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        for at, (args, out, ws, _) in enumerate(calls):
            nt.nt_tree_attention(*args, out, ws, stream=streams[at % 3])
    torch.cuda.synchronize()
    for _, out, ws, want in calls:
        assert nt.nt_workspace_status(ws) == nt.NT_OK and torch.equal(out, want)
    for args, _, ws, want in calls:  # the queries' own place
        q = args[0].clone()
        nt.nt_tree_attention(q, *args[1:], q, ws)
        assert torch.equal(q, want)


@pytest.mark.parametrize("V", [5000, 5001])
def test_adjust_in_place(V):
    rs = np.random.RandomState(V)
    B = 37
    x = (rs.randn(B, V) * 4).astype(np.float32)
    counts = (rs.rand(V) < 0.1).astype(np.int32) * 2
    bias = rs.randn(V).astype(np.float32)
    full = np.tile(counts, (B, 1))
    want = _tree.adjust(x, full, 1.2, 0.5, 0.25, bias, None, np.float32)
    y = dev(x)
    arg = torch.empty(B, dtype=torch.int32, device=DEV)
    ws = torch.zeros(nt.nt_logits_adjust_workspace_size(V, B), dtype=torch.uint8, device=DEV)
    nt.nt_logits_adjust(y, counts=dev(counts), repetition=1.2, frequency=0.5, presence=0.25, bias=dev(bias), out=y, argmax=arg, ws=ws)
    assert np.array_equal(host(y), want) and np.array_equal(host(arg), _tree.choice(want))


def test_a_whole_pass_on_another_stream_and_in_a_graph():
    rs = np.random.RandomState(5)
    B, Hq, Hkv, D, P, V = 12, 8, 2, 128, 300, 3001
    p = _tree.parents(rs, B)
    sees = _tree.ancestors(p)
    side = torch.cuda.Stream()
    q, k, v = (torch.randn(B, h, D, device=DEV) for h in (Hq, Hkv, Hkv))
    kc, vc = (torch.randn(Hkv, P + B, D, device=DEV).bfloat16() for _ in range(2))
    kc0, vc0 = f64(kc), f64(vc)
    parent, token = dev(p), dev(rs.permutation(V)[:B].astype(np.int32))
    mask, pos = torch.zeros(B, 1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    f = torch.zeros(D // 2, dtype=torch.float64, device=DEV)
    qr, out = torch.zeros(B, Hq, D, device=DEV), torch.zeros(B, Hq, D, device=DEV)
    logits, adj = torch.randn(B, V, device=DEV), torch.zeros(B, V, device=DEV)
    am, emit, path = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    n, counts = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(V, dtype=torch.int32, device=DEV)
    ws = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hq, Hkv, D, P), dtype=torch.uint8, device=DEV)
    ws2 = torch.zeros(nt.nt_logits_adjust_workspace_size(V, B), dtype=torch.uint8, device=DEV)
    kp, vp = nt.pointer_array([kc]), nt.pointer_array([vc])

    def step():
        nt.nt_rope_frequencies(D, 1e4, f)
        nt.nt_tree_layout(parent, mask, pos, P)
        nt.nt_qk_norm_rope_append(q, k, v, None, None, 1e-6, f, 0, 1.0, qr, kc, vc, pos=pos, row0=P)
        nt.nt_tree_attention(qr, kc, vc, P, P, mask, out, ws)
        nt.nt_logits_adjust(logits, counts=counts, tree_mask=mask, tokens=token, repetition=1.5, out=adj, argmax=am, ws=ws2)
        nt.nt_tree_accept(parent, token, am, emit, path, n)
        nt.nt_tree_commit(kp, vp, Hkv, D, P + B, path, n, P, P)
        nt.nt_token_counts(token, counts, index=path, n=n)

    wpos = P - 1 + sees.sum(1)
    ff = 1e4 ** (-np.arange(D // 2) * 2.0 / D)
    wq, wk = (_tree.rotate(f64(t), None, 0, ff, 0, 1.0, wpos) for t in (q, k))
    kk, vv = kc0.copy(), vc0.copy()
    kk[:, P:] = f64(torch.from_numpy(wk).float().bfloat16().transpose(0, 1))
    vv[:, P:] = f64(v.bfloat16().transpose(0, 1))
    want = _tree.attend(wq, kk, vv, P, P, sees)
    tk, lg = host(token), host(logits)

    def check(before):
        # a key next to a border of bf16 may round the other way: one product of a score moves by 2^-8
        within(f64(out), want, 2e-2 * np.abs(vv).max(), "out")
        cnt = np.tile(before.astype(np.int64), (B, 1))
        for b in range(B):
            cnt[b, tk[sees[b]]] += 1
        wl = _tree.adjust(lg, cnt, 1.5, 0.0, 0.0, None, None, np.float32)
        assert np.array_equal(host(am), _tree.choice(wl)) and np.array_equal(host(adj), wl)
        wp, we = _tree.accept(p, tk, host(am))
        assert int(n) == len(wp) and host(path).tolist()[:len(wp)] == wp and host(emit).tolist()[:len(wp)] == we
        after = before.copy()
        after[tk[wp]] += 1
        assert np.array_equal(host(counts), after)
        return after

    zero = np.zeros(V, dtype=np.int32)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    check(zero)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (out, am, n, qr, adj, counts):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    after = check(zero)
    graph.replay()
    torch.cuda.synchronize()
    check(after)
