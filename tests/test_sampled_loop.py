"""SampledLoop's checks, against a stand-in for the model (CPU)."""
import types

import pytest

import moe_decode_megakernel_02_gb300 as mk
from moe_decode_megakernel_02_gb300 import sampling


def _model(vocab=100, check=lambda: None):
    return types.SimpleNamespace(config=types.SimpleNamespace(vocab=vocab), check=check)


@pytest.mark.parametrize("vocab", [99, 101, 0])
def test_a_vocabulary_that_is_not_the_models_is_refused(vocab):
    """The step writes the model's vocab logits a row: fewer columns would be written past."""
    with pytest.raises(ValueError):
        sampling.SampledLoop(_model(), None, [1, 2], [0, 0], vocab, device="cpu")
    assert sampling.SampledLoop(_model(), None, [1, 2], [0, 0], 100, device="cpu").tokens() == [[], []]


def test_a_failed_step_stays_failed():
    """Reading the status clears it: tokens drawn after a failed step must not pass for good ones at the next call."""
    codes = [mk.ERR_INVALID_ARG]

    def check():
        if codes:
            raise mk.MKError(codes.pop(), "token id or position out of range for this step")

    loop = sampling.SampledLoop(_model(check=check), None, [1], [0], 100, device="cpu")
    for call in (loop.tokens, loop.tokens, loop.step):
        with pytest.raises(mk.MKError):
            call()
