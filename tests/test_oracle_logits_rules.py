"""Pins of the logits-rules oracle on hand-worked rows."""
import numpy as np

from oracle import logits_rules as L


def test_counts():
    c = np.zeros((3, 5), np.uint16)
    c[2, 1] = 0x7FFE
    tok = np.array([[1, 1, 4, -1], [1, 1, 1, 7]])
    out, bad = L.counts_add(c, tok, lens=np.array([4, 3]), slots=np.array([0, 2]))
    assert not bad
    assert out[0].tolist() == [0, 2, 0, 0, 1] and out[2, 1] == 0x7FFF
    out, bad = L.counts_add(out, tok, lens=np.array([9, 4]), slots=np.array([0, 2]), prompt=True)
    assert bad and out[0].tolist() == [0, 0x8002, 0, 0, 0x8001] and out[2, 1] == 0xFFFF
    assert L.counts_add(c, tok, slots=np.array([3, 0]))[1]


def test_rules_by_hand():
    z = np.array([[[2.0, -2.0, 1.0, 0.0, 3.0], [2.0, -2.0, 1.0, 0.0, 3.0]]])
    rec = np.array([[0x8000, 2, 0, 0, 0]], np.uint16)
    out = L.process(z, counts=rec, path=np.array([[2, 2]]), repetition=[2.0], frequency=[0.5], presence=[0.25],
                    bias_ids=np.array([[3, 3, -1]]), bias=np.array([[1.0, 2.0, 9.0]]))
    # id 0: prompt only; id 1: emitted twice; id 3: bias 1 + 2; row 1 also follows id 2
    np.testing.assert_allclose(out[0, 0], [1.0, -4.0 - 1.0 - 0.25, 1.0, 3.0, 3.0])
    np.testing.assert_allclose(out[0, 1], [1.0, -5.25, 0.5 - 0.5 - 0.25, 3.0, 3.0])
    m = np.array([[[0b00010], [0]]], np.int32)
    out = L.process(np.array([[[np.nan, 1.0], [1.0, 1.0]]]), mask=m)
    assert np.isneginf(out[0, 0, 0]) and out[0, 0, 1] == 1.0 and np.all(np.isneginf(out[0, 1]))
