"""The 8-bit linear and its input gradient give the same bits every time: K-splits of a cluster meet in rank order and no
sum depends on which CTA comes first. The sizes take the cluster, the one-CTA and the CTA-pair forms."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,r", [(9, 4096, 1024, 128), (77, 1040, 1000, 24), (300, 2048, 4096, 0), (2048, 1024, 8192, 64)])
def test_the_same_call_gives_the_same_bits(M, K, N, r):
    import torch
    import sampling_gated_lora_b200 as U
    g = torch.Generator(device="cuda").manual_seed(M)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x = rn(M, K).bfloat16()
    Wq, Ws = U.fp8_quantize((rn(N, K) * K ** -0.5).bfloat16(), 128)
    A, Bl = ((rn(r, K) * K ** -0.5).bfloat16(), rn(N, r).bfloat16()) if r else (None, None)
    gate = (rn(M) > 0).to(torch.uint8)
    y = U.gated_lora_linear_fp8(x, Wq, Ws, A, Bl, gate, 0.5)
    Wqt = Wq.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)
    Wst = Ws.t().contiguous()
    dx = U.gated_lora_input_grad_fp8(y, Wqt, Wst, A, Bl, gate, 0.5) if N % 16 == 0 else None
    for _ in range(8):
        assert torch.equal(U.gated_lora_linear_fp8(x, Wq, Ws, A, Bl, gate, 0.5), y)
        if dx is not None:
            assert torch.equal(U.gated_lora_input_grad_fp8(y, Wqt, Wst, A, Bl, gate, 0.5), dx)
