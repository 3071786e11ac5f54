"""The beam-search example over the numbers of beams that its command takes."""
import pytest

from examples import beam_search as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beams,tokens", [(1, 300), (4, 6), (11, 5), (30, 4), (64, 3)])
def test_the_command_runs(beams, tokens, capsys):
    ex.main(["--beams", str(beams), "--tokens", str(tokens)])
    assert capsys.readouterr().out.count("log probability") == 3


def test_more_beams_than_the_model_was_made_for_are_refused():
    model = ex.PagedDecoder(most=4, n_pages=64)
    with pytest.raises(ValueError, match="at most 4"):
        ex.search(model, [[1, 2], [3]], 3, 2, eos=5)
    with pytest.raises(ValueError, match="must have tokens"):
        ex.search(model, [[1, 2], []], 2, 2, eos=5)
