"""The device error word: a wait that ran out is reported as before, beside an index out of range too."""
import pytest
import torch

import sparse_moe_layer_gb300 as moe


@pytest.mark.gpu
def test_codes_of_the_error_word():
    moe.build()
    for bits, code in ((0, 0), (1, 5), (2, 5), (4, 5), (7, 5), (8, 6), (9, 5), (12, 5)):
        word = moe.new_status()
        word[0] = bits
        assert moe.read_device_status(word) == code, bits
        assert moe.read_device_status(word) == 0
