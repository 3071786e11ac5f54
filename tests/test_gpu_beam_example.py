"""The beam-search example: it runs, its scores are those of scoring its lines from scratch, and neither the page size nor compaction
in between changes what it finds."""
import numpy as np
import pytest
import torch

from examples.beam_search import PagedDecoder, search

pytestmark = pytest.mark.gpu


def scored(model, prompt, line):
    """Log probability of a line behind its prompt, fed as one prompt."""
    model.refs.zero_()
    model.pages, model.length = model.pages[:0], model.length[:0]
    model.fork(model.ints([-1]))
    total, text = 0.0, prompt + line
    logits = model.feed(model.ints(prompt), [len(prompt)])
    for t in text[len(prompt):]:
        total += float(torch.log_softmax(logits[0].double(), 0)[t])
        logits = model.feed(model.ints([t]), [1])
    return total


def test_beams_are_what_their_lines_score():
    rs = np.random.RandomState(0)
    small, large = PagedDecoder(most=12, seed=1), PagedDecoder(most=12, page=64, n_pages=64, seed=1)
    prompts = [rs.randint(0, small.V, n).tolist() for n in (40, 3, 17)]
    a = search(small, prompts, 4, 12, eos=5)
    assert a == search(large, prompts, 4, 12, eos=5)
    assert a == search(small, prompts, 4, 12, eos=5, compact_every=3)
    for prompt, found in zip(prompts, a):
        assert len({tuple(line) for line, _ in found}) == 4, "beams that are alike"
        for line, score in found[:2]:
            # int8 activations: a rounding in the fp32 sums of another order may move a code, 2^-7 of an activation
            assert abs(scored(small, prompt, line) - score) <= 2.0 ** -7 * max(1.0, abs(score)) * len(line)


def test_a_pool_that_is_too_small_says_so():
    model = PagedDecoder(most=4, n_pages=8, seed=0)
    with pytest.raises(RuntimeError, match="no page left"):
        search(model, [[1, 2, 3]], 4, 64, eos=model.V - 1)
