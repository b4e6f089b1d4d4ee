"""Dropout's kernel against the words that its generator's authors published: an element is kept at
p = word / 2^32 and dropped at (word + 1) / 2^32, which fixes all 32 bits of its word."""
import pytest
import torch

import block_reference as ref
from helpers import ensure_built
from test_dropout_words import KNOWN

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbp():
    ensure_built()
    import linear_bound_propagation_amd as m
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=str)
def test_words(lbp, dtype):
    x = torch.ones(1, 4, dtype=dtype, device="cuda")
    for i, word in enumerate(KNOWN[0][2]):
        assert float(lbp.dropout(x, word / 2 ** 32, 0)[0, i]) > 0
        assert float(lbp.dropout(x, (word + 1) / 2 ** 32, 0)[0, i]) == 0
    # other rows, keys and offsets: the integers' form, which the published words pin
    seed, offset = 0x299F31D0A4093822, 0x0370734413198A2E
    x = torch.ones(3, 11, dtype=dtype, device="cuda")
    for r in range(3):
        for c in range(11):
            word = ref.philox((3 * r + c // 4, 0, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0))[c % 4]
            assert float(lbp.dropout(x, word / 2 ** 32, seed, offset)[r, c]) > 0, (r, c)
            assert float(lbp.dropout(x, (word + 1) / 2 ** 32, seed, offset)[r, c]) == 0, (r, c)
