"""Outputs of more than 2^31 elements: offsets past 32 bits in the 8-bit linear and the logits rules."""
import pytest

from test_gpu_fp8 import _case, _dev, _near, _ref

pytestmark = pytest.mark.gpu


def test_linear_output_past_2_31_elements():
    import sampling_gated_lora_b200 as U
    M, K, N, r = 16400, 128, 131072, 8
    assert M * N > 2 ** 31
    x, codes, Ws, A, Bl, gate = _case(M, K, N, r, seed=1)
    y = U.gated_lora_linear_fp8(*_dev(x, codes, Ws, A, Bl, gate), 0.75)
    for rows in (slice(0, 3), slice(M - 20, M)):
        _near(y[rows], *_ref(x[rows], codes, Ws, A, Bl, gate[rows], 0.75), str(rows))


@pytest.mark.parametrize("V", [151936, 151935])
def test_logits_rows_past_2_31_elements(V):
    """One path token a row, in place: that id alone moves, by the frequency penalty (exact in bf16)."""
    import torch
    import sampling_gated_lora_b200 as U
    B = 14200
    assert B * V > 2 ** 31
    z = torch.ones(B, 1, V, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(V)
    path = torch.randint(0, V, (B, 1, 1), generator=g, device="cuda", dtype=torch.int32)
    path[-1] = V - 1
    U.logits_process(z, out=z, draft=path, frequency=torch.full((B,), 0.5, device="cuda"))
    at = z.gather(2, path.long())
    assert bool((at == 0.5).all())
    z.scatter_(2, path.long(), 1.0)
    assert all(bool((part == 1.0).all()) for part in z.split(1000))
    assert U.device_status(clear=True) == 0
