"""The oracle of the conditions on logits, by hand (no GPU)."""

import numpy as np

from oracle import logits as OL


def test_a_row_by_hand():
    h = OL.History(6)
    h.start([1, 1, 9, -1])
    h.add([2, 2, 3, 7])
    assert h.words().tolist() == [0, 0x8000, 2, 1, 0, 0]
    x = np.array([1.0, 2.0, -3.0, 4.0, 5.0, 6.0])
    y = OL.row(x, h, [4, 2, -1], 2.0, 0.5, 0.25, [(0, 1.0), (0, 0.5), (8, 3.0)], np.array([1, 1, 1, 1, 1, 0], bool))
    #          bias    prompt       twice and once more        once       in the row only   not allowed
    assert y.tolist() == [2.5, 1.0, -6.0 - 0.5 - 0.75, 2.0 - 0.75, 2.5 - 0.75, -np.inf]
    assert np.array_equal(OL.row(x, None, [1], 2.0, 1.0, 1.0, [], None), x)
    h.add([2] * 40000)
    assert h.words()[2] == 32767
