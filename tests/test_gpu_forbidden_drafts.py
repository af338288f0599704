"""A drafted id that is masked (-inf) in the AR row is never emitted, whatever the draft row gives it: with p(d) = 0 the
test u q(d) < p(d) fails for q(d) = 0 too. With q(d) = 0 < p(d) it holds for every u."""
import numpy as np
import pytest

import workloads as W
from oracle import sampling as S
from oracle import tree as TR
from gpu_util import TIE_U, compare_drafts, compare_verify, dev_tensor
from test_gpu_empty_rows import FORMS, SEED, STEP, _enc, _same_rows, _verify
from test_gpu_vocab_parallel import _run_sharded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    import sampling_gated_lora_b200 as U
    U.device_status(clear=True)   # the word is the library's: other tests leave bits in it


@pytest.mark.parametrize("form,dtype,V", FORMS)
def test_an_id_masked_in_both_rows_is_rejected(form, dtype, V):
    B, k = 5, 3
    p, q, d = _same_rows(B, k, V, seed=V + 5)
    p[1, 1, d[1, 1]] = q[1, 1, d[1, 1]] = -np.inf
    p[2, 0, d[2, 0]] = q[2, 0, d[2, 0]] = -np.inf
    q[2, 0] = W.bf16_to_f64(W.bf16_round(q[2, 0] + np.linspace(-1, 1, V)))   # the replacement comes from max(p - q, 0)
    half = V // 2 // 8 * 8
    p[3, 2, half:] = q[3, 2, half:] = -np.inf     # all of the upper shard
    d[3, 2] = V - 1
    q[4, 1, d[4, 1]] = -np.inf                    # q = 0 < p: accepted
    want = S.psi_verify(p, q, d, 1.0, SEED, STEP)
    assert want["accepted_len"].tolist() == [k, 1, 0, 2, k]
    acc, tok, cnt, st = _verify(form, p, q, d, dtype)
    assert st == 0
    _, wrong = compare_verify((acc, tok, cnt), want, k, range(B))
    assert not wrong
    for b in range(B):
        assert np.isfinite(p[b, np.arange(cnt[b]), tok[b, :cnt[b]]]).all()


@pytest.mark.parametrize("dtype,V", [("bf16", 1000), ("f32", 4099)])
def test_a_tree_with_forbidden_candidates(dtype, V):
    """Candidates 0 and 2 start with an id that p and q give nothing; candidate 1 starts with an allowed one."""
    import sampling_gated_lora_b200 as U
    B, N, k = 6, 3, 2
    rng = np.random.default_rng(V)
    cands = rng.integers(V // 2, V, (B, N, k)).astype(np.int32)
    cands[:, :, 0] = np.array([V - 3, V // 2 + 1, V - 2])
    p, q, _ = _same_rows(B, N * k, V, seed=V)     # N k + 1 node rows
    q = q[:, :k].copy()
    on = np.zeros(V, bool)
    on[V // 2: V - 3] = True
    p, q = np.where(on, p, -np.inf), np.where(on, q, -np.inf)
    out = U.tree_verify(_enc(p, dtype), _enc(q, dtype), dev_tensor(cands, "i32"), 1.0, SEED, STEP, bonus=True)
    acc, tok, cnt = (t.cpu().numpy() for t in out)
    assert U.device_status() == 0
    for b in range(B):
        nodes = TR.trie(cands[b])[1].shape[0]
        ref = TR.tree_verify_sequence(p[b, :nodes], q[b], cands[b], 1.0, SEED, STEP, b, bonus=True)
        assert on[tok[b, :cnt[b]]].all()
        if ref["test_margin"] > 1e-4 and ref["draw_margin"] > 1e-5:
            assert acc[b] == ref["accepted_len"] and tok[b, :cnt[b]].tolist() == ref["tokens"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shards_that_hold_nothing_but_masked_ids(dtype):
    """Verification and draft over four shards of which one or three are masked whole, against the unsharded oracle."""
    import torch
    from sampling_gated_lora_b200 import vocab_parallel as VPD
    B, k, V, G = 6, 3, 20000, 4
    p, q, _ = _same_rows(B, k, V, seed=77)
    q += 0.5 * np.sin(np.arange(V))
    if dtype == "bf16":
        q = W.bf16_to_f64(W.bf16_round(q))
    else:
        q = q.astype(np.float32).astype(np.float64)
    bounds = VPD.shard_bounds(V, G)
    for b in range(B):   # shard b % 4 alone is left, or left out
        v0, v1 = bounds[b % G]
        on = np.zeros(V, bool)
        on[v0:v1] = True
        if b >= G:
            on = ~on
        p[b], q[b] = np.where(on, p[b], -np.inf), np.where(on, q[b], -np.inf)
    d = S.draft_sample(q, 1.0, 5, 1).astype(np.int32)
    want = S.psi_verify(p, q, d, 1.0, SEED, STEP)
    P, Q, D = _enc(p, dtype), _enc(q, dtype), dev_tensor(d, "i32")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rank_fn(rank, comm):
        v0, v1 = bounds[rank]
        ps, qs = P[..., v0:v1].contiguous(), Q[..., v0:v1].contiguous()
        out = VPD.psi_verify_sharded(ps, qs, D, V, 1.0, SEED, STEP, comm, dev_status=word)
        dn = VPD.draft_sample_sharded(qs, V, 1.0, SEED, STEP, comm, dev_status=word)
        torch.cuda.synchronize()
        return [t.cpu().numpy() for t in (*out, dn)]

    for acc, tok, cnt, dn in _run_sharded(G, rank_fn):
        _, wrong = compare_verify((acc, tok, cnt), want, k, range(B))
        assert not wrong
        _, wrong = compare_drafts(dn, q, 1.0, SEED, STEP)
        assert not wrong
    assert int(word) == 0


@pytest.mark.parametrize("form,dtype,V", FORMS)
def test_ids_below_the_range_of_float_weights(form, dtype, V):
    """Logits so far apart that p(d) and q(d) are below 2^-149, both finite: u < p / q decides, as for any other id (the
    64-bit oracle holds them). A masked one among them is rejected."""
    B, k = 48, 3
    rng = np.random.default_rng(V)
    p = rng.standard_normal((B, k + 1, V)) * 12 - 150
    p[:, :, 0] = 40.0
    q = p[:, :k] + rng.standard_normal((B, k, V))
    q[:, :, 0] = 40.0
    p, q = (W.bf16_to_f64(W.bf16_round(a)) for a in (p, q))
    d = rng.integers(1, V, (B, k)).astype(np.int32)
    p[-1, 1, d[-1, 1]] = q[-1, 1, d[-1, 1]] = -np.inf
    want = S.psi_verify(p, q, d, 1.0, SEED, STEP)
    ratios = np.array([w["ratio"] for w in want["diags"]])
    assert 20 < (want["accepted_len"] > 0).sum() < B and (ratios < 0.5).any() and want["accepted_len"][-1] <= 1
    acc, tok, cnt, st = _verify(form, p, q, d, dtype)
    assert st == 0
    ties = 0
    for b in range(B):
        n = int(acc[b])
        if n != want["accepted_len"][b]:
            j = min(n, int(want["accepted_len"][b]))
            assert abs(want["diags"][b]["u_accept"][j] - ratios[b, j]) < TIE_U
            ties += 1
        # behind the accepted prefix: p(0) = q(0) = 1 up to 2^-200 and every other max(p - q, 0) is below 2^-149, so the
        # residual is 0 in float (the 64-bit oracle still draws from it) and the rule draws from p
        assert tok[b, :n].tolist() == d[b, :n].tolist() and tok[b, n] == 0 and cnt[b] == n + 1
    assert ties <= 1
