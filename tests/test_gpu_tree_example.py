"""The tree-verify calls together, as examples/tree_verify.py uses them: decoding with drafted trees gives
the tokens of decoding one by one, in fewer passes."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed,repetition", [(0, 1.0), (1, 1.0), (2, 1.05)])
def test_drafted_trees_decode_what_single_tokens_decode(seed, repetition):
    from examples import tree_verify as ex
    model = ex.Decoder(seed=seed)
    prompt = np.random.RandomState(seed).randint(0, model.V, 40).tolist()
    one, n_one = ex.generate(model, prompt, 64, tree=False, repetition=repetition)
    many, n_many = ex.generate(model, prompt, 64, tree=True, repetition=repetition)
    assert one == many and n_one == 64
    assert n_many <= n_one
