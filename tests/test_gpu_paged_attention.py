"""Paged attention on the GPU against a plain implementation in 64 bits."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests import _paged
from tests._gpu import DEV, dev

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
I32 = torch.int32


def ints(a):
    return dev(np.ascontiguousarray(a, dtype=np.int32))


def workspace(T, S, Hq, Hkv, D):
    return torch.zeros(nt.nt_paged_attention_workspace_size(T, S, Hq, Hkv, D), dtype=torch.uint8, device=DEV)


class Call:
    """Sequences "new+before" over a pool with random pages; rows that no sequence uses hold NaN."""

    def __init__(self, seqs, Hq, Hkv, D, page, dtype, seed=0, window=0, cap=0.0, slopes=False, spare_tokens=0, scale=1.5, max_new=None,
                 stride=0):
        rs = np.random.RandomState(seed)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.counts, before = (list(x) for x in zip(*[tuple(int(y) for y in s.split("+")) for s in seqs.split()]))
        self.table, self.length, refs = _paged.pool_state(rs, [n + b for n, b in zip(self.counts, before)], page, spare=3)
        self.page, self.window, self.cap, self.Hq, self.Hkv, self.D = page, window, cap, Hq, Hkv, D
        self.T = max(1, sum(self.counts)) + spare_tokens
        wide = torch.randn(self.T, Hq * D + stride, generator=g, device=DEV) * scale
        self.q = wide.to(TYPES[dtype])[:, :Hq * D].view(self.T, Hq, D) if not stride else wide.to(TYPES[dtype])[:, :Hq * D].unflatten(1, (Hq, D))
        rows = len(refs) * page
        self.k, self.v = (torch.full((Hkv, rows, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        for s, n in enumerate(self.length):
            if n:
                at = torch.from_numpy(_paged.rows_of(self.table[s], n, page)).to(DEV)
                for x in (self.k, self.v):
                    x[:, at] = torch.randn(Hkv, n, D, generator=g, device=DEV).bfloat16()
        self.slopes = 2.0 ** (-8.0 * (torch.arange(Hq, device=DEV) + 1.0) / Hq) if slopes else None
        self.max_new = max(self.counts) if max_new is None else max_new
        self.ws = workspace(self.T, len(self.counts), Hq, Hkv, D)
        self.start = ints(np.concatenate(([0], np.cumsum(self.counts))))

    def run(self, out=None, n_bad=None, table=None):
        out = torch.full((self.T, self.Hq, self.D), -7.0, dtype=self.q.dtype, device=DEV) if out is None else out
        nt.nt_paged_attention(self.q, self.k, self.v, self.page, ints(self.table) if table is None else table, self.start, ints(self.length), out,
                              self.ws, max_new=self.max_new, window=self.window, cap=self.cap, slopes=self.slopes, n_bad=n_bad)
        return out

    def want(self):
        return _paged.attend(self.q, self.k, self.v, self.table, self.counts, self.length, self.page, self.window, self.cap, self.slopes)

    def check(self, out, n=None):
        """A score's error: sqrt(D) roundings of |q| |k| / sqrt(D) (half a step or a truncation: 2 U32 each), the cap's or the bias's few
        relative to their size; a weight's is that, twice (its own and the sum's), and its own roundings: 2^-17 in two terms (fp32
        queries), half a step of bf16 (bf16 queries), both in the sum too. Sums lose 2^-16 (fp32) or 2^-12 of the sum of
        |weight| |value| at the very most; the output is rounded once."""
        T = sum(self.counts)
        want, size = self.want()
        want, size, got = want[:T], size[:T], out[:T].double()
        assert (out[T:] == -7.0).all(), "tokens behind the last sequence"
        f32 = self.q.dtype == torch.float32
        clean = lambda x: x.double().nan_to_num(0, 0, 0)  # noqa: E731
        score = float(clean(self.q).norm(dim=-1).max() * clean(self.k).norm(dim=-1).max()) / self.D ** 0.5
        if self.slopes is not None:
            score += float(self.slopes.max()) * float(self.length.max()) / self.D ** 0.5
        x = 2 * 2 * U32 * (self.D ** 0.5 * score + 16 + 4 * self.cap) + (2 * 2.0 ** -17 + 2.0 ** -16 if f32 else 2 * U16 + 2.0 ** -12)
        tol = x * size + (2 * U32 if f32 else U16) * want.abs() + 1e-30
        assert torch.equal(torch.isfinite(want), torch.isfinite(got)), "non-finite outputs elsewhere"
        err = (got - want).abs().nan_to_num(0, 0, 0)
        bad = ~(err <= tol.nan_to_num(torch.inf))
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(err.max())}, first at {bad.nonzero()[0].tolist()}"
        assert int.from_bytes(bytes(self.ws[:4].tolist()), "little") == 0
        return want


SHAPES = ["1+0", "1+1", "1+62", "1+63", "1+64", "1+500 1+0 1+17 1+2000", "2+0", "3+100 1+5 2+63", "1+4094", "0+5 1+9 0+0", "7+30 1+300",
          "33+0", "64+64", "65+63 1+1", "127+129 0+3 5+0", "128+0 129+1", "300+700 1+900 20+0", "513+5"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,page", [(1, 1, 16), (8, 2, 32), (5, 1, 64), (16, 8, 256), (24, 3, 128), (64, 1, 16)])
@pytest.mark.parametrize("seqs", SHAPES)
def test_attention(seqs, Hq, Hkv, page, D, dtype):
    c = Call(seqs, Hq, Hkv, D, page, dtype, seed=len(seqs) + Hq, spare_tokens=Hq % 3)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,cap,slopes", [(1, 0.0, False), (63, 0.0, False), (64, 30.0, False), (100, 0.0, True), (0, 50.0, True), (0, 0.5, False),
                                               (5000, 5.0, True)])
@pytest.mark.parametrize("seqs,Hq,Hkv", [("1+300 1+0 1+77", 8, 2), ("40+200 1+3 1+900", 4, 1), ("260+100", 8, 2), ("129+700 9+0", 3, 3)])
def test_caps_windows_and_slopes(seqs, Hq, Hkv, window, cap, slopes, D, dtype):
    c = Call(seqs, Hq, Hkv, D, 16, dtype, seed=window, window=window, cap=cap, slopes=slopes)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [2.0 ** -100, 1e-20, 1e-3, 255.0, 257.0])
def test_small_and_large_caps(cap, dtype):
    c = Call("70+200 1+3 1+900", 4, 1, 64, 16, dtype, seed=5, cap=cap)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [1e5, 1e12, 2.0 ** 100])
def test_a_cap_far_above_the_scores_loses_nothing_of_them(cap, dtype):
    """cap tanh(x / cap) is off x by at most |x|^3 / (3 cap^2), which is less than a rounding of x here: the tolerance of no cap holds."""
    c = Call("70+200 1+3 1+900", 4, 1, 64, 16, dtype, seed=5, cap=cap)
    score = float(c.q.float().norm(dim=-1).max() * c.k.float().nan_to_num(0).norm(dim=-1).max()) / c.D ** 0.5
    assert score ** 2 / (3 * cap ** 2) < U32
    out = c.run()
    c.cap = 0.0
    c.check(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs,Hq,Hkv,D", [("1+20000", 8, 2, 128), ("1+9000 1+12 1+4000", 32, 8, 64), ("200+9000", 8, 2, 128), ("700+3000 400+0", 4, 1, 64),
                                           ("17+33000", 2, 1, 128), ("1+0 " * 40 + "1+700 " * 40, 8, 2, 128)])
def test_long_sequences_and_many(seqs, Hq, Hkv, D, dtype):
    c = Call(seqs, Hq, Hkv, D, 32, dtype, seed=3)
    a = c.run()
    c.check(a)
    assert torch.equal(a, c.run()), "parts join in the same order every time"


@pytest.mark.parametrize("n", [1, 2, 5, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_number_of_new_tokens(n, dtype):
    c = Call(f"{n}+{3 * n % 200} 1+40", 3, 1, 64, 16, dtype, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_new", [0, 1, 2, 3, 1000])
def test_the_bound_on_new_tokens_only_chooses_the_kernel(max_new, dtype):
    c = Call("1+100 9+20 40+300 1+1 130+0", 4, 2, 64, 16, dtype, max_new=max_new)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs", ["1+70 1+5", "50+70 1+5", "200+10"])
def test_queries_any_stride_apart_and_in_place(seqs, dtype):
    c = Call(seqs, 4, 2, 128, 32, dtype, stride=2 * 128 * 2)
    c.check(c.run())
    c = Call(seqs, 4, 2, 128, 32, dtype)
    want = c.run()
    q = c.q.clone()
    c.q = q
    assert torch.equal(c.run(out=q), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("seqs,window", [("3+20", 0), ("1+100 40+60", 0), ("150+70", 0), ("150+70", 40), ("300+5", 17), ("4+90", 9), ("2+0", 1)])
def test_values_that_are_not_finite_reach_only_those_that_see_them(seqs, window, bad, dtype):
    c = Call(seqs, 4, 2, 64, 16, dtype, window=window, seed=2)
    s = len(c.counts) - 1
    n, length = c.counts[s], int(c.length[s])
    # a value of a late token, and one of an early token that the window has left behind
    for at, d in ((length - 1 - n // 3, 5), (max(0, length - n), 60)):
        c.v[1, int(_paged.rows_of(c.table[s], length, c.page)[at]), d] = bad
    out = c.run()
    want = c.check(out)
    # Which of NaN and infinity comes out is not said: a weight in two terms p = a + b with b < 0 gives a * inf + b * inf = inf - inf
    # where p * inf is infinite.
    assert torch.isfinite(want).any() and not torch.isfinite(want).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs", ["3+20", "150+70", "40+0"])
def test_keys_that_are_not_finite_reach_only_those_that_see_them(seqs, dtype):
    c = Call(seqs, 4, 2, 64, 16, dtype)
    n, length = c.counts[0], int(c.length[0])
    c.k[0, int(_paged.rows_of(c.table[0], length, c.page)[length - n // 2 - 1])] = float("nan")
    out = c.run()
    want = c.check(out)
    assert torch.isfinite(want[:n - n // 2 - 1]).all() and torch.isnan(want[-1, 0]).all() and torch.isfinite(want[-1, -1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_tokens_that_see_nothing(n, dtype):
    c = Call(f"{n}+10 {n}+3", 4, 2, 64, 16, dtype)
    c.length[0] = n // 2  # fewer rows than new tokens: the first ones stand before the sequence
    c.length[1] = 0
    out = c.run()
    c.check(out)
    assert (out[:n - n // 2] == 0).all() and (out[n:2 * n] == 0).all()
    c.length[1] = -5
    assert (c.run()[n:2 * n] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs", ["1+70", "60+70", "180+70"])
def test_pages_out_of_range_read_as_zeros_and_are_counted(seqs, dtype):
    c = Call(seqs, 4, 2, 64, 16, dtype)
    n_bad = torch.zeros(1, dtype=I32, device=DEV)
    c.run(n_bad=n_bad)
    assert int(n_bad) == 0
    good = c.table.copy()
    for page in (len(c.k[0]) // 16, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 27):
        table = good.copy()
        table[0, 2] = page
        n_bad.zero_()
        out = c.run(n_bad=n_bad, table=ints(table))
        assert int(n_bad) > 0
        keep = c.k.clone(), c.v.clone()
        at = _paged.rows_of(good[0], 48, 16)[32:]
        c.k[:, at], c.v[:, at] = 0.0, 0.0
        c.check(out)
        c.k, c.v = keep


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 50])
def test_rows_behind_the_last_sequence_and_starts_out_of_range(n, dtype):
    c = Call(f"{n}+20 {n}+3", 4, 2, 64, 16, dtype, spare_tokens=13)
    c.check(c.run())
    c.start = ints([-3, n, 2 * n])
    c.check(c.run())
    c.start = ints([0, n, 10 ** 9])  # cut to T: the second sequence has 13 more tokens
    out = c.run()
    c.counts[1] += 13
    c.check(out)


def test_offsets_beyond_32_bits():
    """A pool of 2^31 elements a head and more: the sequence's pages stand at its end."""
    D, page, Hkv = 128, 256, 2
    rows = (1 << 31) // D + 4 * page
    k, v = (torch.zeros(Hkv, rows, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for n, dtype in ((1, torch.float32), (70, torch.float32), (70, torch.bfloat16), (300, torch.bfloat16)):
        last = rows // page - 1
        table, length = np.array([[last, last - 1, last - 2]], dtype=np.int32), np.array([600], dtype=np.int32)
        at = _paged.rows_of(table[0], 600, page)
        for x in (k, v):
            x[:, at] = torch.randn(Hkv, 600, D, device=DEV).bfloat16()
        q = torch.randn(n, 4, D, device=DEV).to(dtype)
        out = torch.empty_like(q)
        nt.nt_paged_attention(q, k, v, page, ints(table), ints([0, n]), ints(length), out, workspace(n, 1, 4, Hkv, D), max_new=n)
        lo = int(at.min())
        want, size = _paged.attend(q, k[:, lo:], v[:, lo:], table - lo // page, [n], length, page)
        assert lo % page == 0
        tol = size * (2.0 ** -14 if dtype == torch.float32 else 2.0 ** -6)
        assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_and_flat_scores(dtype):
    c = Call("5+90 60+200 1+300", 4, 2, 128, 16, dtype, scale=40.0)
    c.check(c.run())
    c.k.fill_(0.25)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rise", "fall", "one sign"])
@pytest.mark.parametrize("seqs", ["1+3000", "40+3000", "200+6000"])
def test_scores_that_rise_and_sums_of_one_sign(seqs, kind, dtype):
    """The reference maximum moves with every tile; sums of values of one sign, where cut-off bits add up."""
    c = Call(seqs, 2, 1, 64, 64, dtype)
    length = int(c.length[0])
    at = torch.from_numpy(_paged.rows_of(c.table[0], length, 64)).to(DEV)
    if kind == "one sign":
        c.v[:, at] = c.v[:, at].abs() + 1.0
        c.k[:, at] *= 0.05
    else:
        ramp = torch.linspace(0.0, 3.0, length, device=DEV)
        c.q = c.q.abs()
        c.k[:, at] = (ramp if kind == "rise" else ramp.flip(0))[None, :, None].expand(1, length, 64).bfloat16()
    c.check(c.run())


@pytest.mark.parametrize("seqs", ["1+300 1+7 1+1000", "70+300 1+7 33+0"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths_change_between_replays_of_a_graph(seqs, dtype):
    """On a stream of its own; the tables, lengths and starts of the replay count, not the recording's."""
    c = Call(seqs, 8, 2, 128, 16, dtype)
    d = Call("1+100 2+40 1+900" if seqs.startswith("1+") else "50+301 40+100 1+50", 8, 2, 128, 16, dtype, seed=5)
    stream = torch.cuda.Stream()
    T, W, rows = max(c.T, d.T), max(c.table.shape[1], d.table.shape[1]), max(c.k.shape[1], d.k.shape[1])
    q, out = torch.zeros(T, 8, 128, dtype=c.q.dtype, device=DEV), torch.zeros(T, 8, 128, dtype=c.q.dtype, device=DEV)
    k, v = (torch.zeros(2, rows, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table, length, start = torch.zeros(3, W, dtype=I32, device=DEV), torch.zeros(3, dtype=I32, device=DEV), torch.zeros(4, dtype=I32, device=DEV)
    ws = workspace(T, 3, 8, 2, 128)

    def load(x):
        out.fill_(-7.0)
        q[:x.T] = x.q
        k[:, :x.k.shape[1]], v[:, :x.v.shape[1]] = x.k, x.v
        table[:, :x.table.shape[1]] = ints(x.table)
        length.copy_(ints(x.length))
        start.copy_(x.start)

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        load(c)
        step = lambda: nt.nt_paged_attention(q, k, v, 16, table, start, length, out, ws, max_new=70 if c.max_new > 2 else 2)  # noqa: E731
        step()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
        for x in (d, c, d):
            load(x)
            for _ in range(3):
                g.replay()
            stream.synchronize()
            got = torch.full((x.T, 8, 128), -7.0, dtype=c.q.dtype, device=DEV)
            got[:sum(x.counts)] = out[:sum(x.counts)]
            x.check(got)


def test_agrees_with_the_attention_of_one_sequence():
    """Chains of new tokens over one contiguous sequence: pages in order are nt_attention_decode's cache."""
    for B, before in ((1, 200), (5, 1000), (16, 77)):
        n = before + B
        k, v = (torch.randn(2, 2048, 128, device=DEV).bfloat16() for _ in range(2))
        q = torch.randn(B, 8, 128, device=DEV)
        a, b = torch.empty_like(q), torch.empty_like(q)
        ws = torch.zeros(nt.nt_attention_workspace_size(B, 8, 2, n), dtype=torch.uint8, device=DEV)
        nt.nt_attention_decode(q, k, v, B, 8, 2, 128, n, 2048, a, ws)
        nt.nt_paged_attention(q, k, v, 16, ints(np.arange(128)[None]), ints([0, B]), ints([n]), b, workspace(B, 1, 8, 2, 128), max_new=B)
        assert ((a - b).abs() <= 2.0 ** -14 * float(v.float().abs().max())).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", ["40+300", "300+5000 1+40"])
def test_a_wait_that_runs_out_is_reported_until_the_workspace_is_cleared(seqs, D, dtype):
    """No copies are issued (a host-side hook): the waits end after 20 ms, nothing hangs."""
    c = Call(seqs, 4, 2, D, 32, dtype)
    try:
        nt.nt_set_test_fault(6, 20.0)
        c.run()
        torch.cuda.synchronize()
    finally:
        nt.nt_set_test_fault(0)
    assert nt.nt_workspace_status(c.ws) == nt.NT_ERR_TIMEOUT
    c.ws.zero_()
    c.check(c.run())
    assert nt.nt_workspace_status(c.ws) == nt.NT_OK


@pytest.mark.parametrize("n", [2, 64])
def test_starts_that_do_not_rise_do_no_harm(n):
    """What comes out is not said; nothing is written outside the outputs."""
    c = Call(" ".join([f"{n}+40"] * 6), 8, 2, 64, 16, "f32", max_new=n)
    c.start = ints([0, 6 * n, 0, 6 * n, 0, 6 * n, 0])
    c.run()
    c.start = ints([6 * n, 5, 4, 3, 2, 1, 0])
    c.run()
    torch.cuda.synchronize()
    c.ws.zero_()
    c.start = ints(np.arange(7) * n)
    c.check(c.run())
