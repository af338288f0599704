"""The repetition penalty divides: with no other rule on, a float logit of a prompt id comes out as the quotient
z / repetition rounded once (z > 0) or the product (z <= 0), bit for bit, and a bf16 one as that quotient in float rounded
to bf16 (the reciprocal's own rounding, 2^-24, would show only where a quotient lies that near to the middle of two bf16
values; none here does)."""
import numpy as np
import pytest

import workloads as W
from gpu_util import dev_tensor

pytestmark = pytest.mark.gpu

TINY = np.float32(2.0 ** -140)   # its reciprocal is no float
RHOS = [1.3, 0.7, 1.0, 3.0, 1e-30, 3e38, TINY]


def _prompt_of(V):
    """Every other id in the prompt; id 0 is reached through the path below."""
    c = np.zeros((len(RHOS), V), np.uint16)
    c[:, 1::2] = 0x8000
    return c


@pytest.mark.parametrize("V", [1000, 1001, 1004])
def test_quotients_are_rounded_once(V):
    import torch
    import sampling_gated_lora_b200 as U
    rng = np.random.default_rng(V)
    B = len(RHOS)
    rho = np.array(RHOS, np.float32)
    z = (rng.standard_normal((B, 2, V)) * 3).astype(np.float32)
    z *= np.minimum(rho, 1)[:, None, None]   # small ones by small factors
    c = torch.from_numpy(_prompt_of(V).view(np.int16)).cuda()
    path = np.zeros((B, 1), np.int32)      # row 1 follows id 0
    with np.errstate(all="ignore"):
        held = np.broadcast_to((_prompt_of(V) != 0)[:, None], z.shape).copy()
        held[:, 1, 0] = True
        ref = np.where(held, np.where(z > 0, z / rho[:, None, None], z * rho[:, None, None]), z).astype(np.float32)
    got = U.logits_process(dev_tensor(z, "f32"), counts=c, draft=dev_tensor(path, "i32"), repetition=dev_tensor(rho, "f32"))
    np.testing.assert_array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("V", [1000, 1001])
def test_bf16_quotients(V):
    import torch
    import sampling_gated_lora_b200 as U
    rng = np.random.default_rng(V)
    B = len(RHOS)
    rho = np.array(RHOS, np.float32)
    zb = W.bf16_round(rng.standard_normal((B, 1, V)) * 3 * np.minimum(rho, 1).astype(np.float64)[:, None, None])
    z = W.bf16_to_f64(zb).astype(np.float32)
    c = torch.from_numpy(_prompt_of(V).view(np.int16)).cuda()
    with np.errstate(all="ignore"):
        q = np.where((_prompt_of(V) != 0)[:, None], np.where(z > 0, z / rho[:, None, None], z * rho[:, None, None]), z)
    want = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    got = U.logits_process(dev_tensor(zb, "bf16"), counts=c, repetition=dev_tensor(rho, "f32")).cpu()
    assert torch.equal(got, want)


@pytest.mark.parametrize("V", [1000, 1001])
@pytest.mark.parametrize("rho", [2.0 ** -126, 1.9 * 2.0 ** -126, 2.0 ** 127.5])
def test_bf16_quotients_by_the_smallest_and_largest_factors(rho, V):
    """z of the factor's size, so that the quotients are ordinary numbers."""
    import torch
    import sampling_gated_lora_b200 as U
    rng = np.random.default_rng(V)
    rho = np.float32(rho)
    zb = W.bf16_round(rng.uniform(1.0, 2.0, (1, 1, V)) * max(float(rho) / 2, 2.0 ** -126))
    z = W.bf16_to_f64(zb).astype(np.float32)
    want = torch.from_numpy(z / rho).to(torch.bfloat16)
    c = torch.full((1, V), -32768, dtype=torch.int16, device="cuda")
    got = U.logits_process(dev_tensor(zb, "bf16"), counts=c, repetition=dev_tensor(rho.reshape(1), "f32")).cpu()
    assert bool(torch.isfinite(want).all()) and torch.equal(got, want)
