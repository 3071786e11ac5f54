"""bf16 results of chunks are as exact as rounding allows: nothing but the output's own rounding shows."""
import pytest

from tests.test_gpu_paged_attention import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(window=300), dict(slopes=True)], ids=["all", "window", "bias"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", ["40+700", "120+3000 1+500", "600+0", "300+1000 33+90 1+20"])
def test_only_the_outputs_rounding_shows(seqs, D, kw):
    """The root of the mean square error next to that of rounding the exact result. Weights of two terms add 2^-17 of a step of 2^-8 and
    sums cut off 2^-13 of sums of random signs, less than a hundredth in the square; weights of one rounded term are off by as much as the output's
    rounding, which makes it 1.2 to 1.4."""
    c = Call(seqs, 8, 2, D, 32, "bf16", **kw)
    out = c.run()
    want = c.check(out)[:sum(c.counts)]
    error, rounding = ((x.double() - want).pow(2).mean().sqrt() for x in (out[:sum(c.counts)], want.bfloat16()))
    assert float(error / rounding) <= 1.02
