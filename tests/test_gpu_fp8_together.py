"""The 8-bit linear, the logits rules and the token records together with the framework's own calls, as a program
uses them: decode steps (gated head over 8-bit weights, rules, draft, verification, records) and one training pass
(two gated layers, distillation, adapter gradients, input gradient)."""
import numpy as np
import pytest

import workloads as W
from oracle import distill as D
from oracle import fp8
from oracle import logits_rules as L
from oracle import sampling as S
from oracle.gated_linear import gated_linear_adapter_grads
from gpu_util import check_verify_outputs_valid, compare_drafts, compare_verify, dev_tensor, host_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    import sampling_gated_lora_b200 as U
    U.device_status(clear=True)   # the word is the library's: other tests leave bits in it


def _fp8_weight(rng, N, K):
    import sampling_gated_lora_b200 as U
    return U.fp8_quantize(dev_tensor(W.bf16_round(rng.standard_normal((N, K)) * K ** -0.5 * 3), "bf16"), 128)


def test_decode_steps_under_rules():
    """Three steps of 6 sequences: the AR rows follow the drafted prefix, both paths share the records, the biases
    and each sequence's mask; what is emitted is allowed and lands in the records."""
    import torch
    import sampling_gated_lora_b200 as U
    B, k, V, K, r = 6, 3, 1208, 256, 16
    rng = np.random.default_rng(0)
    bf = lambda *s, std=1.0: dev_tensor(W.bf16_round(rng.standard_normal(s) * std), "bf16")   # noqa: E731
    Wq, Ws = _fp8_weight(rng, V, K)
    A, Bl = bf(r, K, std=K ** -0.5), bf(V, r, std=0.1)
    rows_p, rows_q = B * (k + 1), B * k
    gate = torch.cat([torch.zeros(rows_p), torch.ones(rows_q)]).to(torch.uint8).cuda()
    words = (V + 31) // 32
    on = rng.random((B, 32 * words)) < np.where(np.arange(B)[:, None] % 2, 0.05, 1.0)
    on[:, 7] = True
    mask = np.packbits(on, axis=-1, bitorder="little").view(np.int32)
    rules = dict(repetition=np.full(B, 1.2, np.float32), frequency=np.full(B, 0.3, np.float32),
                 presence=np.full(B, 0.2, np.float32), bias_ids=rng.integers(0, V, (B, 4)).astype(np.int32),
                 bias=np.full((B, 4), 2.0, np.float32))
    dev = {n: dev_tensor(a, "i32" if a.dtype == np.int32 else "f32") for n, a in rules.items()}
    prompts = rng.integers(0, V, (B, 20)).astype(np.int32)
    slots = np.array([4, 2, 7, 0, 1, 5], np.int32)
    counts = torch.zeros(8, V, dtype=torch.int16, device="cuda")
    U.token_counts_add(counts, dev_tensor(prompts, "i32"), slots=dev_tensor(slots, "i32"), prompt=True)
    ref_counts, _ = L.counts_add(np.zeros((8, V), np.uint16), prompts, slots=slots, prompt=True)
    work = torch.empty(U.gated_lora_linear_fp8_workspace(rows_p + rows_q, K, V, r), dtype=torch.uint8, device="cuda")
    mrows = lambda n: np.repeat(mask[:, None], n, 1)   # noqa: E731
    q_prev = d_prev = None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(4):
        h = bf(rows_p + rows_q, K)
        z = U.gated_lora_linear_fp8(h, Wq, Ws, A, Bl, gate, 1.0, workspace=work)
        p, q = z[:rows_p].view(B, k + 1, V), z[rows_p:].view(B, k, V)
        raw_p, raw_q = host_f64(p), host_f64(q)
        if d_prev is not None:
            U.logits_process(p, out=p, counts=counts, slots=dev_tensor(slots, "i32"), draft=d_prev,
                             mask=dev_tensor(mrows(k + 1), "i32"), dev_status=status, **dev)
            path = d_prev.cpu().numpy()
            want = L.process(raw_p, ref_counts, slots, path, mask=mrows(k + 1), **rules)
            got = host_f64(p)
            f = np.isfinite(want)
            np.testing.assert_array_equal(np.isfinite(got), f)
            # half a bf16 step, and 2^-20 for the float additions before it (terms below 16)
            assert np.all(np.abs(got[f] - want[f]) <= 2.0 ** -8 * np.abs(want[f]) + 2.0 ** -20)
            acc, tok, cnt = U.psi_verify(p, q_prev, d_prev, 1.0, 11, step, dev_status=status)
            out = [t.cpu().numpy() for t in (acc, tok, cnt)]
            check_verify_outputs_valid(*out, path, k, k + 1, V)
            ora = S.psi_verify(got, host_f64(q_prev), path, 1.0, 11, step)
            _, bad = compare_verify(out, ora, k, range(B))
            assert not bad
            for b in range(B):
                assert on[b, out[1][b, :out[2][b]]].all()
            U.token_counts_add(counts, tok, slots=dev_tensor(slots, "i32"), dev_status=status)
            ref_counts, _ = L.counts_add(ref_counts, out[1], slots=slots)
            np.testing.assert_array_equal(counts.cpu().numpy().view(np.uint16), ref_counts)
        q_prev = U.logits_process(q, counts=counts, slots=dev_tensor(slots, "i32"), mask=dev_tensor(mrows(k), "i32"), **dev)
        d_prev = U.draft_sample(q_prev, 1.0, 11, step)
        _, bad = compare_drafts(d_prev.cpu().numpy(), host_f64(q_prev), 1.0, 11, step)
        assert not bad and on[np.arange(B)[:, None], d_prev.cpu().numpy()].all()
    assert int(status) == 0 and U.device_status() == 0


def test_rules_on_tree_nodes():
    """A candidate tree's node rows with each node's own path: a token the path holds is penalised there only."""
    import torch
    import sampling_gated_lora_b200 as U
    B, N, k, V = 2, 3, 2, 512
    rng = np.random.default_rng(3)
    R = N * k + 1
    cands = rng.integers(0, V, (B, N, k)).astype(np.int32)
    path = np.full((B, R, k), -1, np.int32)
    for b in range(B):   # three disjoint blocks: node 1 + i k + j holds candidate i's first j + 1 tokens
        cands[b, :, 0] = [1, 2, 3]
        for i in range(N):
            for j in range(k):
                path[b, 1 + i * k + j, :j + 1] = cands[b, i, :j + 1]
    z = W.bf16_round(rng.standard_normal((B, R, V)) * 3)
    p = U.logits_process(dev_tensor(z, "bf16"), draft=dev_tensor(path, "i32"),
                         frequency=dev_tensor(np.full(B, 4.0), "f32"))
    want = L.process(W.bf16_to_f64(z), path=path, frequency=np.full(B, 4.0))
    got = host_f64(p)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want))
    assert np.array_equal(got != W.bf16_to_f64(z), want != W.bf16_to_f64(z))
    q = dev_tensor(W.bf16_round(rng.standard_normal((B, k, V))), "bf16")
    acc, tok, cnt = U.tree_verify(p, q, dev_tensor(cands, "i32"), 1.0, 5, 0)
    assert U.device_status() == 0 and torch.all(cnt == acc + (acc < k))


def test_training_pass_over_8_bit_layers():
    """Forward through two gated layers, distillation against a teacher, gradients back to both adapters; every call
    is held to the oracle on the operands it was given."""
    import sampling_gated_lora_b200 as U
    M, K, H, V, r = 48, 256, 384, 528, 16
    rng = np.random.default_rng(5)
    bf = lambda *s, std=1.0: dev_tensor(W.bf16_round(rng.standard_normal(s) * std), "bf16")   # noqa: E731
    W1, s1 = _fp8_weight(rng, H, K)
    W2, s2 = _fp8_weight(rng, V, H)
    A1, B1, A2, B2 = bf(r, K, std=K ** -0.5), bf(H, r, std=0.1), bf(r, H, std=H ** -0.5), bf(V, r, std=0.1)
    gate = dev_tensor(np.ones(M), "u8")
    x, teacher = bf(M, K), bf(M, V)
    h = U.gated_lora_linear_fp8(x, W1, s1, A1, B1, gate, 1.0)
    z = U.gated_lora_linear_fp8(h, W2, s2, A2, B2, gate, 1.0)
    losses, dz = U.distill(teacher, z, alpha=1.0, beta=0.5)
    dzb = (dz * 64).bfloat16()
    u8 = lambda t: t.view(__import__("torch").uint8)   # noqa: E731
    f8 = x.new_empty(0, dtype=W2.dtype).dtype
    W2t = u8(W2).t().contiguous().view(f8)
    dA2, dB2 = U.gated_lora_adapter_grads(h, dzb, A2, B2, gate, 1.0)
    dh = U.gated_lora_input_grad_fp8(dzb, W2t, s2.t().contiguous(), A2, B2, gate, 1.0)
    dA1, dB1 = U.gated_lora_adapter_grads(x, dh, A1, B1, gate, 1.0)

    c2 = fp8.code_values()[u8(W2).cpu().numpy()]
    g = np.ones(M)
    n = lambda t: host_f64(t)   # noqa: E731
    y, bound = fp8.gated_linear_fp8(n(h), c2, s2.cpu().numpy(), n(A2), n(B2), g, 1.0)
    assert np.all(np.abs(n(z) - y) <= bound)
    want, bound = fp8.gated_input_grad_fp8(n(dzb), c2, s2.cpu().numpy(), n(A2), n(B2), g, 1.0)
    assert np.all(np.abs(n(dh) - want) <= bound)
    for got, ref in zip((dA2, dB2, dA1, dB1), gated_linear_adapter_grads(n(h), n(A2), n(B2), g, 1.0, n(dzb))
                        + gated_linear_adapter_grads(n(x), n(A1), n(B1), g, 1.0, n(dh))):
        rms = np.sqrt(np.mean(ref * ref))
        assert rms > 0 and np.all(np.abs(n(got) - ref) <= 3e-2 * rms + 2.0 ** -8 * np.abs(ref))
    kl, tv = D.distill_losses(n(teacher), n(z), 1.0)
    np.testing.assert_allclose(losses.cpu().numpy(), np.stack([kl, tv], 1), rtol=1e-3, atol=1e-5)
