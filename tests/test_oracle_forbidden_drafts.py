"""Pins of the accept test at q(d) = 0: an id that p gives nothing is rejected, by the linear, the tree and the sharded
verification; one that p gives something is accepted. Shards that are masked whole weigh nothing."""
from fractions import Fraction

import numpy as np

from oracle import sampling as S
from oracle import tree as TR
from oracle import vocab_parallel as VP


def test_threshold():
    assert S.accept_threshold(Fraction(0), Fraction(0)) == 0 and S.accept_threshold(0.0, 0.0) == 0
    assert S.accept_threshold(Fraction(1, 9), Fraction(0)) == 1 and S.accept_threshold(Fraction(0), Fraction(1, 9)) == 0


def _case():
    rng = np.random.default_rng(3)
    p = rng.standard_normal((4, 3, 40))
    q = p[:, :2].copy()
    d = S.draft_sample(q, 1.0, 1, 0)
    p[1, 0, d[1, 0]] = q[1, 0, d[1, 0]] = -np.inf     # in neither row
    p[2, 1, d[2, 1]] = -np.inf                        # in q only
    q[3, 1, d[3, 1]] = -np.inf                        # in p only
    return p, q, d


def test_linear_and_sharded():
    p, q, d = _case()
    out = S.psi_verify(p, q, d, 1.0, 5, 0)
    assert out["accepted_len"].tolist() == [2, 0, 1, 2]
    assert out["out_tokens"][1, 0] != d[1, 0] and out["out_tokens"][2, 1] != d[2, 1]
    p[0, :, :16] = q[0, :, :16] = -np.inf             # the first shard of sequence 0
    d[0] = S.draft_sample(q[:1], 1.0, 1, 0)[0]
    want = S.psi_verify(p, q, d, 1.0, 5, 0)
    bounds = VP.shard_bounds(40, 3)
    assert bounds[0] == (0, 16)
    got = VP.vp_psi_verify(VP.split(p, bounds), VP.split(q, bounds), bounds, d, 1.0, 5, 0)
    for key in ("accepted_len", "out_tokens", "out_count"):
        np.testing.assert_array_equal(got[key], want[key])
    np.testing.assert_array_equal(VP.vp_draft_sample(VP.split(q, bounds), bounds, 1.0, 5, 0),
                                  S.draft_sample(q, 1.0, 5, 0))


def test_tree():
    rng = np.random.default_rng(4)
    p = rng.standard_normal((3, 12))
    q = p[:1].copy()
    p[:, 5] = q[:, 5] = -np.inf
    r = TR.tree_verify_sequence(p, q, np.array([[5], [7]]), 1.0, 2, 0, 0)
    assert r["accepted_len"] == 1 and r["tokens"] == [7]
