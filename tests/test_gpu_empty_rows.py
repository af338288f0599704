"""Rows of logits without a distribution (nothing but -inf, or a NaN) in verification: a sequence that needs one is
reported (outputs -1, UNO_DEV_NAN) by every form of the call, and its output buffers hold nothing from before."""
import numpy as np
import pytest

import workloads as W
from oracle import sampling as S
from gpu_util import compare_verify, dev_tensor
from test_gpu_vocab_parallel import _run_sharded

pytestmark = pytest.mark.gpu

SEED, STEP = 9, 4


@pytest.fixture(autouse=True)
def _clean_status():
    import sampling_gated_lora_b200 as U
    U.device_status(clear=True)   # the word is the library's: other tests leave bits in it


def _same_rows(B, k, V, seed):
    """AR and draft logits that agree at the k drafted positions (every draft is accepted), in bf16 values."""
    lc = W.logits_case(B, k, V, k_p=k + 1, ar_std=3.0, sigma=0.0, seed=seed)
    p = W.bf16_to_f64(lc.p_logits).reshape(B, k + 1, V)
    q = p[:, :k].copy()
    return p, q, S.draft_sample(q, 1.0, seed, 0).astype(np.int32)


def _enc(a, dtype):
    return dev_tensor(W.bf16_round(a) if dtype == "bf16" else a, dtype)


def _verify(form, p, q, d, dtype):
    """(accepted_len, out_tokens, out_count, status) of one form of the call; buffers start as 12345."""
    import torch
    import sampling_gated_lora_b200 as U
    from sampling_gated_lora_b200 import vocab_parallel as VPD
    B, k, V = q.shape
    P, Q, D = _enc(p, dtype), _enc(q, dtype), dev_tensor(d, "i32")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if form == "sharded":
        bounds = VPD.shard_bounds(V, 2)

        def rank_fn(rank, comm):
            v0, v1 = bounds[rank]
            out = VPD.psi_verify_sharded(P[..., v0:v1].contiguous(), Q[..., v0:v1].contiguous(), D, V, 1.0, SEED, STEP,
                                         comm, dev_status=st)
            torch.cuda.synchronize()
            return [t.cpu().numpy() for t in out]
        res = _run_sharded(2, rank_fn)
        for a, b in zip(*res):
            np.testing.assert_array_equal(a, b)
        return (*res[0], int(st))
    full = lambda *s: torch.full(s, 12345, dtype=torch.int32, device="cuda")   # noqa: E731
    buf = dict(accepted_len=full(B), out_tokens=full(B, k + 1), out_count=full(B), dev_status=st)
    if form == "tree":
        out = U.tree_verify(P, Q, D[:, None].contiguous(), 1.0, SEED, STEP, bonus=True, **buf)
    elif form == "noalloc":
        out = U.psi_verify_noalloc(P, Q, D, 1.0, SEED, STEP, **buf)
    else:
        out = U.psi_verify(P, Q, D, 1.0, SEED, STEP, **buf)
    return (*(t.cpu().numpy() for t in out), int(st))


FORMS = [("linear", "bf16", 1000), ("linear", "bf16", 1001), ("linear", "f32", 20000), ("linear", "bf16", 151936),
         ("noalloc", "bf16", 1000), ("tree", "bf16", 1001), ("tree", "f32", 20000), ("sharded", "bf16", 20000),
         ("sharded", "f32", 1000)]


@pytest.mark.parametrize("what", [-np.inf, np.nan])
@pytest.mark.parametrize("form,dtype,V", FORMS)
def test_a_bonus_row_without_a_distribution_is_reported(form, dtype, V, what):
    import sampling_gated_lora_b200 as U
    B, k = 4, 3
    p, q, d = _same_rows(B, k, V, seed=V)
    want = S.psi_verify(p, q, d, 1.0, SEED, STEP)
    assert np.all(want["accepted_len"] == k)   # so the bonus row of every sequence is read
    bad = p.copy()
    if np.isnan(what):
        bad[1, k, V // 2] = what
    else:
        bad[1, k] = what
    acc, tok, cnt, st = _verify(form, bad, q, d, dtype)
    assert st == U.DEV_NAN and acc[1] == -1 and cnt[1] == -1 and np.all(tok[1] == -1)
    _, wrong = compare_verify((acc, tok, cnt), want, k, [0, 2, 3])
    assert not wrong


@pytest.mark.parametrize("form,dtype,V", FORMS)
def test_rows_behind_the_first_rejection_may_be_empty(form, dtype, V):
    """A drafted id leaves the grammar (p = 0 there) and the AR rows behind it, the bonus row among them, allow nothing:
    the accepted prefix and its replacement token come out as with any other rows there."""
    B, k = 4, 3
    p, q, d = _same_rows(B, k, V, seed=V + 1)
    p[1, 1, d[1, 1]] = -np.inf    # rejected at position 1
    p[2, 0, d[2, 0]] = -np.inf    # at position 0
    want = S.psi_verify(p, q, d, 1.0, SEED, STEP)
    assert want["accepted_len"].tolist() == [k, 1, 0, k]
    bad = p.copy()
    bad[1, 2:] = bad[2, 1:] = -np.inf
    acc, tok, cnt, st = _verify(form, bad, q, d, dtype)
    assert st == 0
    _, wrong = compare_verify((acc, tok, cnt), want, k, range(B))
    assert not wrong


@pytest.mark.parametrize("form,dtype,V", FORMS)
def test_empty_rows_up_to_the_first_rejection_are_reported(form, dtype, V):
    import sampling_gated_lora_b200 as U
    B, k = 4, 3
    p, q, d = _same_rows(B, k, V, seed=V + 2)
    p[1, 2, d[1, 2]] = -np.inf
    p[1, 1] = -np.inf             # needed before the rejection at position 2
    p[2, 0] = -np.inf             # the first row
    q[3, 1] = -np.inf             # no draft distribution where the block is still accepted
    acc, tok, cnt, st = _verify(form, p, q, d, dtype)
    assert st == U.DEV_NAN and np.all(acc[1:] == -1) and np.all(cnt[1:] == -1) and np.all(tok[1:] == -1)
    assert acc[0] == k


@pytest.mark.parametrize("form,dtype,V", [f for f in FORMS if f[0] != "tree"])   # the walk reads no row behind its end
def test_a_nan_at_any_drafted_position_is_reported(form, dtype, V):
    import sampling_gated_lora_b200 as U
    B, k = 2, 3
    p, q, d = _same_rows(B, k, V, seed=V + 3)
    p[1, 0, d[1, 0]] = -np.inf
    p[1, 2, V - 1] = np.nan
    acc, tok, cnt, st = _verify(form, p, q, d, dtype)
    assert st == U.DEV_NAN and acc[0] == k and acc[1] == -1 and cnt[1] == -1 and np.all(tok[1] == -1)
