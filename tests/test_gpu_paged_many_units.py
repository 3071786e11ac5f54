"""Calls of more sequences, or tiles of rows, than a CTA has threads: the division of the work goes through them in rounds."""
import pytest

from tests.test_gpu_paged_attention import Call

pytestmark = pytest.mark.gpu


def decode(S, most, new=1):
    return " ".join(f"{new}+{(s * 377) % most}" for s in range(S))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [257, 300, 513, 2000, 4096])
def test_many_sequences_of_few_rows(S, dtype):
    c = Call(decode(S, 150), 4, 2, 64, 16, dtype, seed=S)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,Hq,Hkv", [(769, 64, 1), (1600, 64, 1), (3300, 32, 1)])
def test_many_tiles_of_one_chunk(new, Hq, Hkv, dtype):
    c = Call(f"{new}+100", Hq, Hkv, 64, 64, dtype, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [390, 1200])
def test_many_sequences_with_a_tile_each(S, dtype):
    c = Call(decode(S, 200, 9), 4, 2, 64, 16, dtype, seed=2)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_of_both_kinds(dtype):
    seqs = " ".join(f"{(1, 1, 2, 1, 40, 0)[s % 6]}+{(s * 31) % 300}" for s in range(1500)) + " 300+1000"
    c = Call(seqs, 4, 2, 64, 16, dtype, seed=3, spare_tokens=3)
    c.check(c.run())
    c.max_new = 0
    c.check(c.run())
