"""Verification of logits with masked (-inf) ids: whole 16-byte vectors, threads' shares and 8192-id chunks of a row
may hold nothing else. Masked ids have probability 0; a row without a finite logit is reported as before."""
import numpy as np
import pytest

import workloads as W
from oracle import sampling as S
from gpu_util import check_verify_outputs_valid, compare_drafts, compare_verify, dev_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    import sampling_gated_lora_b200 as U
    U.device_status(clear=True)   # the word is the library's: other tests leave bits in it


def _masked(B, k, kp, V, allowed, dtype, seed):
    rng = np.random.default_rng(seed)
    lc = W.logits_case(B, k, V, k_p=kp, ar_std=3.0, sigma=0.5, seed=seed, dtype=dtype)
    f = (lambda a: W.bf16_to_f64(a)) if dtype == "bf16" else (lambda a: np.asarray(a, np.float64))
    p, q = f(lc.p_logits).reshape(B, kp, V), f(lc.q_logits).reshape(B, k, V)
    on = np.zeros((B, V), bool)
    for b in range(B):
        on[b, rng.choice(V, allowed, replace=False)] = True
    p, q = np.where(on[:, None], p, -np.inf), np.where(on[:, None], q, -np.inf)
    return p, q, S.draft_sample(q, 1.0, seed, 0).astype(np.int32), on


def _enc(a, dtype):
    return dev_tensor(W.bf16_round(a) if dtype == "bf16" else a, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,allowed", [(1000, 3), (1001, 1), (20000, 5), (151936, 12), (151936, 140000)])
def test_psi_verify_on_masked_rows(V, allowed, dtype):
    import sampling_gated_lora_b200 as U
    B, k = 6, 3
    p, q, d, on = _masked(B, k, k + 1, V, allowed, dtype, seed=V + allowed)
    out = U.psi_verify(_enc(p, dtype), _enc(q, dtype), dev_tensor(d, "i32"), 1.0, 9, 4)
    acc, tok, cnt = (t.cpu().numpy() for t in out)
    check_verify_outputs_valid(acc, tok, cnt, d, k, k + 1, V)
    _, bad = compare_verify((acc, tok, cnt), S.psi_verify(p, q, d, 1.0, 9, 4), k, range(B))
    assert not bad and U.device_status() == 0
    assert all(on[b, tok[b, :cnt[b]]].all() for b in range(B))
    cands = np.ascontiguousarray(d[:, None])   # one candidate block: the tree walk gives the same tokens
    nodes = np.ascontiguousarray(p)
    t = U.tree_verify(_enc(nodes, dtype), _enc(q, dtype), dev_tensor(cands, "i32"), 1.0, 9, 4, bonus=True)
    same = [np.array_equal(a.cpu().numpy(), b) for a, b in zip(t, (acc, tok, cnt))]
    assert all(same) and U.device_status() == 0


def test_a_row_without_a_finite_logit_and_a_nan_among_masked_ones_are_reported():
    import sampling_gated_lora_b200 as U
    B, k, V = 3, 2, 20000
    p, q, d, _ = _masked(B, k, k + 1, V, 50, "f32", seed=2)
    p[1, 0] = -np.inf
    p[2, 1, np.flatnonzero(~np.isfinite(p[2, 1]))[-1]] = np.nan
    acc, tok, cnt = U.psi_verify(_enc(p, "f32"), _enc(q, "f32"), dev_tensor(d, "i32"), 1.0, 9, 4)
    assert U.device_status() & U.DEV_NAN
    assert int(acc[1]) == -1 and int(acc[2]) == -1 and int(acc[0]) >= 0 and (tok[1:] == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,allowed", [(1000, 3), (1001, 1), (20000, 5), (151936, 12), (151936, 140000)])
def test_draft_on_masked_rows(V, allowed, dtype):
    import sampling_gated_lora_b200 as U
    B, k = 6, 3
    _, q, _, on = _masked(B, k, k + 1, V, allowed, dtype, seed=V + allowed)
    d = U.draft_sample(_enc(q, dtype), 1.0, 9, 4).cpu().numpy()
    _, bad = compare_drafts(d, q, 1.0, 9, 4)
    assert not bad and U.device_status() == 0
    assert on[np.arange(B)[:, None], d].all()
