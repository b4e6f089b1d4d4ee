"""The forms of dropout's generator that the other tests and the cases compare with, against the words
that its authors published for seven rounds (Salmon, Moraes, Dror and Shaw, 2011: known answers)."""
import numpy as np
import torch

import block_reference as ref
from perf import more_operators as cases

# counter, key, words
KNOWN = [((0, 0, 0, 0), (0, 0), (0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48)),
         ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662)),
         ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
          (0x4DFCCABA, 0x190A87F0, 0xC47362BA, 0xB6B5242A))]


def test_integers():
    for counter, key, words in KNOWN:
        assert tuple(ref.philox(counter, key)) == words


def test_masks():
    """The first row's four words decide: kept at p = word / 2^32, dropped one step above."""
    words = KNOWN[0][2]
    for i, word in enumerate(words):
        at, above = word / 2 ** 32, (word + 1) / 2 ** 32
        assert bool(ref.kept(1, 4, at, 0, 0)[0, i]) and not bool(ref.kept(1, 4, above, 0, 0)[0, i])
        assert cases._kept(1, 4, 0, 0, at)[0, i] and not cases._kept(1, 4, 0, 0, above)[0, i]
    assert tuple(cases._random_words(1, 4, 0, 0, "cpu")[0].tolist()) == words
    # beyond one row, and with every half of key and counter
    seed, offset = 0x299F31D0A4093822, 0x0370734413198A2E
    got = cases._random_words(3, 6, seed, offset, torch.device("cpu"))
    for r in range(3):
        for c in range(6):
            word = ref.philox((2 * r + c // 4, 0, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0))[c % 4]
            assert int(got[r, c]) == word
            mask = cases._kept(3, 6, seed, offset, word / 2 ** 32)
            assert mask[r, c] and np.array_equal(mask, ref.kept(3, 6, word / 2 ** 32, seed, offset).numpy())
