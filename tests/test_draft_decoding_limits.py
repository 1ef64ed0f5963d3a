"""The example of draft decoding refuses texts past its model's places before anything reaches the GPU."""

import os
import sys
import types

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_texts_past_the_models_places_are_refused():
    import draft_decoding as ex

    class Reached(Exception):
        pass

    def model(*a):
        raise Reached()

    run = ex.Decoder.__new__(ex.Decoder)
    run.model, run.table = types.SimpleNamespace(max_len=16, page=8), None
    with pytest.raises(ValueError, match="16 places"):      # an index past the place embeddings would end the process
        run.forward([[1, 2], [3]], [9, 17], [])
    run.text = [[0] * 14, [0] * 3]
    with pytest.raises(ValueError, match="16 places"):
        run.round(4)
