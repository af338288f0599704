"""8-bit block-scaled quantiser, gated linear and its input gradient on the GPU vs the oracle.

Codes and scales follow a float32 recipe and have to be equal. Products are
held, element by element, to the bound that oracle.fp8.gated_linear_fp8 derives
from fp32 sums, the bf16 rounding of x A^T and the bf16 result."""
import numpy as np
import pytest

import workloads as W
from oracle import fp8
from gpu_util import dev_tensor, host_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    import sampling_gated_lora_b200 as U
    U.device_status(clear=True)   # the word is the library's: other tests leave bits in it


def _codes(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def _bf16(rng, *shape, std=1.0):
    return W.bf16_round(rng.standard_normal(shape) * std)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 128), (9, 4096), (127, 136), (129, 1000), (513, 2048), (1024, 4104)])
def test_quantize_equals_the_recipe(M, K, rows, dtype):
    import sampling_gated_lora_b200 as U
    rng = np.random.default_rng(M * K + rows)
    x = rng.standard_normal((M, K)) * np.exp(4 * rng.standard_normal((M, 1)))
    x[:, : K // 2 : 3] = 0.0
    if M > 4:
        x[3] = 0.0
    xb = W.bf16_round(x) if dtype == "bf16" else x.astype(np.float32)
    xf = W.bf16_to_f64(xb) if dtype == "bf16" else xb
    codes, scales = U.fp8_quantize(dev_tensor(xb, dtype), rows)
    v, s = fp8.quantize(xf, rows)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(fp8.code_values()[_codes(codes)], v)


def test_quantize_marks_blocks_that_are_not_finite():
    import sampling_gated_lora_b200 as U
    x = np.ones((130, 256), np.float32)
    x[1, 5], x[2, 200] = np.nan, np.inf
    x[0, :128] = np.float32(1e-38)
    codes, scales = U.fp8_quantize(dev_tensor(x, "f32"), 1)
    s, v = scales.cpu().numpy(), fp8.code_values()[_codes(codes)]
    assert np.isnan(s[1, 0]) and np.isnan(v[1, :128]).all() and np.isinf(s[2, 1])
    bad = np.zeros_like(s, bool)
    bad[1, 0] = bad[2, 1] = True
    assert np.isfinite(s[~bad]).all() and np.isfinite(np.delete(v, [1, 2], 0)).all()
    _, sb = U.fp8_quantize(dev_tensor(x, "f32"), 128)
    sb = sb.cpu().numpy()
    assert np.isnan(sb[0, 0]) and np.isinf(sb[0, 1]) and np.isfinite(sb[1]).all()


def _case(M, K, N, r, seed, own_scales=False):
    rng = np.random.default_rng(seed)
    x = _bf16(rng, M, K)
    if own_scales:   # any codes under any scales, as a checkpoint brings them
        codes = rng.integers(0, 256, (N, K)).astype(np.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x11
        Ws = np.exp(2 * rng.standard_normal((-(-N // 128), -(-K // 128)))).astype(np.float32) * 1e-3
    else:
        v, Ws = fp8.quantize(W.bf16_to_f64(_bf16(rng, N, K, std=K ** -0.5)), 128)
        table = fp8.code_values()[:127]
        codes = (np.searchsorted(table, np.abs(v)) + 128 * (np.signbit(v))).astype(np.uint8)
    A, Bl = (_bf16(rng, r, K, std=K ** -0.5), _bf16(rng, N, r, std=0.1)) if r else (None, None)
    gate = (rng.random(M) < 0.5).astype(np.uint8)
    return x, codes, Ws, A, Bl, gate


def _dev(x, codes, Ws, A, Bl, gate):
    import torch
    t = lambda a: None if a is None else dev_tensor(a, "bf16")   # noqa: E731
    wq = torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(torch.float8_e4m3fn)
    return t(x), wq, dev_tensor(Ws, "f32"), t(A), t(Bl), dev_tensor(gate, "u8")


def _ref(x, codes, Ws, A, Bl, gate, scale):
    f = lambda a: None if a is None else W.bf16_to_f64(a)   # noqa: E731
    return fp8.gated_linear_fp8(f(x), fp8.code_values()[codes], Ws, f(A), f(Bl), gate, scale)


def _near(y, ref, bound, what):
    err = np.abs(host_f64(y) - ref)
    assert np.all(err <= bound), f"{what}: {np.max(err / np.maximum(bound, 1e-300)):.3f} of the bound"


SHAPES = [
    (1, 16, 8, 0), (1, 128, 128, 8), (5, 16, 16, 8), (150, 16, 8, 200), (2, 144, 136, 16), (9, 1024, 512, 128), (16, 512, 4096, 64),
    (17, 2048, 200, 24), (32, 272, 1000, 256), (33, 1040, 1000, 24), (64, 4096, 384, 128), (65, 640, 256, 8),
    (128, 1024, 1024, 128), (129, 528, 264, 40), (200, 12288, 136, 128), (257, 1024, 520, 16), (300, 144, 2048, 200),
    (577, 1040, 776, 128), (1000, 512, 4096, 128),
    (40, 128, 40064, 256), (300, 128, 20480, 256), (129, 1024, 37888, 8), (5000, 144, 264, 16),   # several tiles a CTA
    (100, 256, 33024, 0), (2500, 272, 2304, 128),
]


@pytest.mark.parametrize("M,K,N,r", SHAPES)
def test_linear_matches_the_oracle(M, K, N, r):
    import sampling_gated_lora_b200 as U
    c = _case(M, K, N, r, seed=M + K + N)
    y = U.gated_lora_linear_fp8(*_dev(*c), 0.75)
    _near(y, *_ref(*c, 0.75), f"{M}x{K}x{N} r={r}")
    assert U.device_status() == 0


@pytest.mark.parametrize("M,K,N,r", [(3, 144, 136, 8), (40, 1040, 264, 0), (150, 400, 640, 32), (700, 272, 520, 16)])
def test_linear_takes_any_codes_and_scales(M, K, N, r):
    import sampling_gated_lora_b200 as U
    c = _case(M, K, N, r, seed=M, own_scales=True)
    _near(U.gated_lora_linear_fp8(*_dev(*c), 1.0), *_ref(*c, 1.0), f"{M}x{K}x{N} r={r}")


@pytest.mark.parametrize("M,K,N,r", [(1, 8, 16, 8), (9, 512, 1024, 128), (33, 1000, 1040, 24), (130, 136, 2048, 0),
                                     (300, 264, 528, 256), (600, 1024, 1040, 64)])
def test_input_gradient_matches_the_oracle(M, K, N, r):
    import torch
    import sampling_gated_lora_b200 as U
    _, codes, Ws, A, Bl, gate = _case(M, 16 * -(-K // 16), N, r, seed=M + N)
    codes, Ws = codes[:, :K], Ws[:, : -(-K // 128)]
    A = None if A is None else np.ascontiguousarray(A[:, :K])
    dy = _bf16(np.random.default_rng(M), M, N, std=1e-3)
    d, wq, ws, a, bl, g = _dev(dy, codes, Ws, A, Bl, gate)
    wqt = wq.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)
    dx = U.gated_lora_input_grad_fp8(d, wqt, ws.t().contiguous(), a, bl, g, 0.5)
    f = lambda z: None if z is None else W.bf16_to_f64(z)   # noqa: E731
    _near(dx, *fp8.gated_input_grad_fp8(f(dy), fp8.code_values()[codes], Ws, f(A), f(Bl), gate, 0.5),
          f"{M}x{K}x{N} r={r}")


def test_gradient_is_what_differences_of_the_output_say():
    """Row by row, <dy, y(x + d) - y(x)> = <dx, d>. x and dy hold exact e4m3 values with a 448 in every block
    (scales 1), and d turns those around, so x and x + d are exact too. What rounds is bf16: y twice, t = x A^T
    twice, u = dy Bl and dx once, each by 2^-8 of its values; 2^-14 covers the fp32 sums (128-deep blocks)."""
    import torch
    import sampling_gated_lora_b200 as U
    M, K, N, r = 24, 256, 384, 16
    rng = np.random.default_rng(4)
    _, codes, Ws, A, Bl, gate = _case(M, K, N, r, seed=4)
    gate[:] = 1

    def draw(*shape):
        v = rng.choice(np.array([-4.0, -2.0, -1.0, 0.0, 1.0, 2.0, 4.0]), shape)
        v[:, ::128] = 448.0
        return v
    x0, dy = draw(M, K), draw(M, N)
    d = np.zeros((M, K))
    d[:, ::128] = -896.0
    args = _dev(W.bf16_round(x0), codes, Ws, A, Bl, gate)
    wqt = args[1].view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn)
    t = lambda v: dev_tensor(W.bf16_round(v), "bf16")   # noqa: E731
    dx = host_f64(U.gated_lora_input_grad_fp8(t(dy), wqt, args[2].t().contiguous(), *args[3:], 0.5))
    y0, y1 = (host_f64(U.gated_lora_linear_fp8(t(v), *args[1:], 0.5)) for v in (x0, x0 + d))
    a, b = W.bf16_to_f64(A), W.bf16_to_f64(Bl)
    ts = sum(np.abs(0.5 * v @ a.T) for v in (x0, x0 + d)) @ np.abs(b).T     # |t| through the up-projection
    us = np.abs(0.5 * dy @ b) @ np.abs(a)                                     # |u| through A
    ay = np.abs(y0) + np.abs(y1)
    tol = (2.0 ** -8 + 2.0 ** -14) * ((np.abs(dy) * (ay + ts)).sum(1) + (np.abs(d) * (np.abs(dx) + us)).sum(1))
    moved, said = (dy * (y1 - y0)).sum(1), (dx * d).sum(1)
    assert np.all(np.abs(moved - said) <= tol)
    assert np.median(np.abs(said) / tol) > 2     # the test can tell


def test_gate_zero_rows_are_the_base_product_and_no_rows_launch_nothing():
    import torch
    import sampling_gated_lora_b200 as U
    x, wq, ws, A, Bl, gate = _dev(*_case(40, 512, 384, 16, seed=3))
    y0 = U.gated_lora_linear_fp8(x, wq, ws, None, None, None)
    y1 = U.gated_lora_linear_fp8(x, wq, ws, A, Bl, torch.zeros_like(gate))
    y2 = U.gated_lora_linear_fp8(x, wq, ws, A, Bl, gate)
    assert torch.equal(y0, y1) and torch.equal(y0[gate == 0], y2[gate == 0])
    assert not torch.equal(y0[gate == 1], y2[gate == 1])
    assert U.gated_lora_linear_fp8(x[:0], wq, ws, A, Bl, gate[:0]).shape == (0, 384)


def test_rows_do_not_depend_on_each_other():
    """A NaN row, an infinite row and rows of zeros leave the others as they are."""
    import torch
    import sampling_gated_lora_b200 as U
    for M in (12, 300):
        x, wq, ws, A, Bl, gate = _dev(*_case(M, 512, 384, 16, seed=M))
        gate.fill_(1)
        y = U.gated_lora_linear_fp8(x, wq, ws, A, Bl, gate)
        z = x.clone()
        z[2, 7], z[5, 300], z[7] = float("nan"), float("inf"), 0.0
        o = U.gated_lora_linear_fp8(z, wq, ws, A, Bl, gate)
        keep = [i for i in range(M) if i not in (2, 5, 7)]
        assert torch.equal(o[keep], y[keep])
        assert o[2].isnan().all() and not o[5].isfinite().any() and not o[7].any()


@pytest.mark.parametrize("M", [9, 150, 600])
def test_graph_replays_streams_and_a_shared_workspace(M):
    """One workspace for calls in order on one stream, captured and replayed on new inputs, with guards
    around the output."""
    import torch
    import sampling_gated_lora_b200 as U
    K, N, r = 1024, 520, 32
    c = _case(M, K, N, r, seed=M)
    x, wq, ws, A, Bl, gate = _dev(*c)
    want = U.gated_lora_linear_fp8(x, wq, ws, A, Bl, gate, 0.75)
    need = U.gated_lora_linear_fp8_workspace(M, K, N, r)
    work = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    big = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    xin = torch.zeros_like(x)
    with torch.cuda.stream(s):
        U.gated_lora_linear_fp8(xin, wq, ws, A, Bl, gate, 0.75, y=big[1:-1], workspace=work)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            U.gated_lora_linear_fp8(xin, wq, ws, A, Bl, gate, 0.75, y=big[1:-1], workspace=work)
        for k in range(3):
            xin.copy_(x if k != 1 else -x)
            g.replay()
            got = big[1:-1].clone()
            assert torch.equal(got, want if k != 1 else -want)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.all(big[0] == 7.0) and torch.all(big[-1] == 7.0)


def test_calls_on_a_stream_given_by_argument():
    """Outputs and workspaces made by the call belong to that stream: two of them run their calls side by side."""
    import torch
    import sampling_gated_lora_b200 as U
    cases = [_dev(*_case(M, 512, 384, 16, seed=M)) for M in (20, 200)]
    want = [U.gated_lora_linear_fp8(*c, 0.75) for c in cases]
    codes = U.fp8_quantize(cases[1][0])[0]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i].append(U.gated_lora_linear_fp8(*cases[i], 0.75, stream=s))
            other = U.fp8_quantize(cases[1][0], stream=s)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys, w in zip(got, want) for y in ys)
    assert torch.equal(other.view(torch.uint8), codes.view(torch.uint8))


def test_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, sampling_gated_lora_b200 as U
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
x, A, Bl, gate = r(9, 256), r(8, 256), r(384, 8), torch.ones(9, dtype=torch.uint8, device="cuda")
Wq = (torch.randn(384, 256, generator=g, device="cuda")).to(torch.float8_e4m3fn)
Ws = torch.full((3, 2), 0.5, device="cuda")
z, y = r(1, 2, 1000), torch.zeros(9, 384, device="cuda", dtype=torch.bfloat16)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    U.gated_lora_linear_fp8(x, Wq, Ws, A, Bl, gate, 1.0, y=y)
    U.logits_process(z, out=z, presence=torch.ones(1, device="cuda"))
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, U.gated_lora_linear_fp8(x, Wq, Ws, A, Bl, gate, 1.0)) and bool(y.any())
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)
