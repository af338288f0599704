"""Refusals of the 8-bit linear, its quantiser, the token records and the logits rules: in the binding (shapes,
types, devices) and in the C ABI (sizes, NULL and unaligned pointers, workspaces, overlaps). No GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import sampling_gated_lora_b200 as U

bf16, f32, i16, i32, u8, f8 = (torch.bfloat16, torch.float32, torch.int16, torch.int32, torch.uint8,
                               torch.float8_e4m3fn)
OK, NULL, ODD = ctypes.c_void_p(0x10000), None, ctypes.c_void_p(0x10008)


def _linear(M=4, K=272, N=136, r=8):
    return dict(x=torch.zeros(M, K, dtype=bf16), Wq=torch.zeros(N, K, dtype=f8), Ws=torch.zeros(2, 3),
                A=torch.zeros(r, K, dtype=bf16), Bl=torch.zeros(N, r, dtype=bf16), gate=torch.zeros(M, dtype=u8))


def test_well_formed_calls_reach_the_device_check():
    with pytest.raises(ValueError, match="CUDA device"):
        U.gated_lora_linear_fp8(**_linear())
    a = _linear()
    with pytest.raises(ValueError, match="CUDA device"):
        U.gated_lora_input_grad_fp8(torch.zeros(4, 136, dtype=bf16), a["Wq"].view(u8).t().contiguous().view(f8),
                                    a["Ws"].t().contiguous(), a["A"], a["Bl"], a["gate"])
    with pytest.raises(ValueError, match="CUDA device"):
        U.fp8_quantize(a["x"])
    with pytest.raises(ValueError, match="CUDA device"):
        U.token_counts_add(torch.zeros(2, 9, dtype=i16), torch.zeros(2, 3, dtype=i32))
    with pytest.raises(ValueError, match="CUDA device"):
        U.logits_process(torch.zeros(1, 2, 9))


@pytest.mark.parametrize("name,bad,err", [
    ("x", torch.zeros(4, 272), TypeError), ("Wq", torch.zeros(136, 256, dtype=f8), ValueError),
    ("Wq", torch.zeros(136, 272, dtype=u8), TypeError), ("Wq", torch.zeros(136, 272, dtype=torch.float8_e5m2), TypeError),
    ("Ws", torch.zeros(2, 2), ValueError), ("Ws", torch.zeros(1, 3), ValueError), ("Ws", torch.zeros(2, 3, dtype=bf16), TypeError),
    ("A", torch.zeros(8, 256, dtype=bf16), ValueError), ("Bl", torch.zeros(136, 4, dtype=bf16), ValueError),
    ("gate", torch.zeros(5, dtype=u8), ValueError), ("gate", None, ValueError), ("Bl", None, ValueError)])
def test_linear_operands(name, bad, err):
    a = _linear()
    a[name] = bad
    with pytest.raises(err, match=name):
        U.gated_lora_linear_fp8(**a)


def test_gradient_and_quantiser_operands():
    a = _linear()
    dy, Wqt, Wst = torch.zeros(4, 136, dtype=bf16), torch.zeros(272, 136, dtype=f8), torch.zeros(3, 2)
    call = lambda **k: U.gated_lora_input_grad_fp8(**{**dict(dy=dy, Wqt=Wqt, Wst=Wst, A=a["A"], Bl=a["Bl"], gate=a["gate"]), **k})  # noqa: E731
    for k, v in (("Wqt", a["Wq"]), ("Wst", a["Ws"]), ("A", a["A"][:, :8]), ("dx", torch.zeros(4, 136, dtype=bf16))):
        with pytest.raises(ValueError, match=k):
            call(**{k: v})
    with pytest.raises(ValueError, match="block_rows"):
        U.fp8_quantize(a["x"], 64)
    with pytest.raises(ValueError, match="scales"):
        U.fp8_quantize(a["x"], 128, scales=torch.zeros(4, 3))
    with pytest.raises(TypeError, match="codes"):
        U.fp8_quantize(a["x"], codes=torch.zeros(4, 272, dtype=u8))


@pytest.mark.parametrize("kw,err,msg", [
    (dict(counts=torch.zeros(2, 8, dtype=i16)), ValueError, "counts"), (dict(counts=torch.zeros(2, 9, dtype=i32)), TypeError, "counts"),
    (dict(slots=torch.zeros(3, dtype=i32)), ValueError, "slots"), (dict(draft=torch.zeros(1, 4, dtype=i32)), ValueError, "draft"),
    (dict(draft=torch.zeros(2, 4, 4, dtype=i32)), ValueError, "draft"), (dict(repetition=torch.zeros(2, dtype=bf16)), TypeError, "repetition"),
    (dict(bias=torch.zeros(2, 4)), ValueError, "bias_ids"), (dict(bias_ids=torch.zeros(2, 4, dtype=i32)), ValueError, "bias"),
    (dict(bias_ids=torch.zeros(2, 4, dtype=i32), bias=torch.zeros(2, 5)), ValueError, "bias"),
    (dict(mask=torch.zeros(2, 3, 2, dtype=i32)), ValueError, "mask"), (dict(out=torch.zeros(2, 3, 9, dtype=bf16)), TypeError, "out")])
def test_logits_operands(kw, err, msg):
    with pytest.raises(err, match=msg):
        U.logits_process(torch.zeros(2, 3, 9), **kw)


def test_counts_operands():
    c, t = torch.zeros(2, 9, dtype=i16), torch.zeros(2, 3, dtype=i32)
    for kw in (dict(lens=torch.zeros(3, dtype=i32)), dict(slots=torch.zeros(1, dtype=i32))):
        with pytest.raises(ValueError):
            U.token_counts_add(c, t, **kw)
    with pytest.raises(TypeError):
        U.token_counts_add(c, t.long())


def test_abi_refuses_bad_8_bit_calls():
    L = U.load()
    q = lambda dt=U.UNO_BF16, M=4, K=136, rows=1, x=OK, c=OK, s=OK: L.uno_fp8_quantize(dt, M, K, rows, x, c, s, NULL)  # noqa: E731
    assert q(dt=5) == 1 and q(M=-1) == 1 and q(K=0) == 1 and q(rows=64) == 1 and q(K=12) == 2
    assert q(x=NULL) == 1 and q(c=NULL) == 1 and q(s=ODD) == 1 and q(M=0, x=NULL) == 0
    for grad in (False, True):
        fn = L.uno_gated_lora_input_grad_fp8 if grad else L.uno_gated_lora_linear_fp8
        wsq = L.uno_gated_lora_input_grad_fp8_workspace if grad else L.uno_gated_lora_linear_fp8_workspace

        def f(dt=U.UNO_BF16, M=4, Kc=144, No=136, r=8, x=OK, W=OK, s=OK, A=OK, B=OK, g=OK, y=OK, ws=OK, n=1 << 30):
            K, N = (No, Kc) if grad else (Kc, No)
            return fn(dt, M, K, N, r, x, W, s, A, B, g, 1.0, y, ws, n, NULL)
        assert f(dt=U.UNO_F32) == 2 and f(M=-1) == 1 and f(Kc=0) == 1 and f(r=-8) == 1
        assert f(Kc=136) == 2 and f(No=132) == 2 and f(r=4) == 2 and f(r=264) == 2 and f(M=(1 << 24) + 1) == 2
        assert f(No=(1 << 23) + 8) == 2
        for k in ("x", "W", "s", "A", "B", "g", "y"):
            assert f(**{k: NULL}) == 1, k
            if k != "g":
                assert f(**{k: ODD}) == 1, k
        assert f(ws=NULL) == 6 and f(ws=ODD) == 6 and f(n=wsq(4, *((136, 144) if grad else (144, 136)), 8) - 1) == 6
        assert f(M=0, x=NULL, ws=NULL) == 0
        assert wsq(-1, 16, 16, 8) == 0 and wsq(4, 0, 16, 8) == 0 and wsq(4, 144, 144, 0) > 4 * 144


def test_abi_refuses_bad_logits_calls():
    L = U.load()
    c = lambda S=2, V=9, cn=OK, B=2, T=3, tok=OK, slots=NULL, prompt=0: L.uno_token_counts_add(  # noqa: E731
        S, V, cn, B, T, tok, NULL, slots, prompt, NULL, NULL)
    assert c(S=-1) == 1 and c(B=-1) == 1 and c(T=-1) == 1 and c(V=1) == 2 and c(V=196609) == 2 and c(prompt=2) == 1
    assert c(cn=NULL) == 1 and c(cn=ODD) == 1 and c(tok=NULL) == 1 and c(S=1) == 1 and c(T=0, tok=NULL) == 0

    def f(dt=U.UNO_BF16, B=2, R=3, V=16, z=OK, o=OK, S=2, cn=NULL, slots=NULL, P=0, pr=0, path=NULL, nb=0, ids=NULL,
          bias=NULL, mask=NULL):
        return L.uno_logits_process(dt, B, R, V, z, o, S, cn, slots, P, pr, path, NULL, NULL, NULL, nb, ids, bias, mask,
                                    NULL, NULL)
    assert f(dt=3) == 1 and f(B=-1) == 1 and f(R=-1) == 1 and f(P=-1) == 1 and f(nb=-1) == 1
    assert f(V=1) == 2 and f(V=200000) == 2 and f(P=65, path=OK) == 2 and f(nb=1025, ids=OK, bias=OK) == 2
    assert f(pr=2) == 1 and f(z=NULL) == 1 and f(o=NULL) == 1 and f(P=2) == 1 and f(nb=2, ids=OK) == 1
    assert f(z=ODD) == 1 and f(mask=ODD) == 1 and f(cn=ODD) == 1 and f(cn=OK, S=1) == 1
    assert f(o=ctypes.c_void_p(0x10010)) == 1 and f(z=ctypes.c_void_p(0x10010)) == 1      # partial overlap
    assert f(B=0, z=NULL) == 0 and f(R=0, z=NULL) == 0
