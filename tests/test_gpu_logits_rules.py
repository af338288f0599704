"""Token records and logits rules on the GPU vs the oracle.

Records are whole numbers and have to be equal. Logits are computed in float
and rounded once: a division, a product, three additions and the sum of at most
nb biases change |z|-sized terms by 2^-24 each, and the result's type rounds by
half a step (bf16 2^-8, float 2^-24)."""
import numpy as np
import pytest

import workloads as W
from oracle import logits_rules as L
from gpu_util import dev_tensor, host_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    import sampling_gated_lora_b200 as U
    U.device_status(clear=True)   # the word is the library's: other tests leave bits in it


def _i16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


@pytest.mark.parametrize("V", [2, 33, 1000, 151936])
@pytest.mark.parametrize("prompt", [False, True])
def test_counts_match_the_oracle(V, prompt):
    import torch
    import sampling_gated_lora_b200 as U
    rng = np.random.default_rng(V)
    for B, T in ((1, 1), (5, 33), (3, 700)):
        S = B + 2
        c = rng.choice(np.array([0, 1, 0x7FFE, 0x7FFF, 0x8000, 0xFFFE], np.uint16), (S, V))
        tok = rng.integers(0, min(V, 40), (B, T)).astype(np.int32)
        tok[rng.random((B, T)) < 0.1] = -1
        lens = rng.integers(-1, T + 3, B).astype(np.int32)
        slots = rng.permutation(S)[:B].astype(np.int32)
        if B > 2:
            slots[1] = slots[0]   # two sequences on one record
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = U.token_counts_add(_i16(c), dev_tensor(tok, "i32"), dev_tensor(lens, "i32"), dev_tensor(slots, "i32"),
                                 prompt, dev_status=st)
        want, bad = L.counts_add(c, tok, lens, slots, prompt)
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint16), want)
        assert int(st) == 0 and not bad


def test_counts_skip_and_report_what_is_out_of_range():
    import torch
    import sampling_gated_lora_b200 as U
    c = np.zeros((2, 10), np.uint16)
    tok = np.array([[1, 10, -2, 3], [4, 4, -1, 2**31 - 1]], np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = _i16(c)
    U.token_counts_add(d, dev_tensor(tok, "i32"), dev_status=st)
    np.testing.assert_array_equal(d.cpu().numpy().view(np.uint16), L.counts_add(c, tok)[0])
    assert int(st) == U.DEV_BAD_INDEX and U.device_status() == U.DEV_BAD_INDEX
    U.token_counts_add(d, dev_tensor(tok[:1], "i32"), slots=dev_tensor(np.array([2]), "i32"))
    assert U.device_status() == U.DEV_BAD_INDEX and int(d.sum()) == 4


def _case(B, R, V, P, nb, tree, seed, allowed=0.3):
    rng = np.random.default_rng(seed)
    S = B + 1
    z = rng.standard_normal((B, R, V)) * 3
    c = np.where(rng.random((S, V)) < 0.02, rng.integers(0, 5, (S, V)), 0).astype(np.uint16)
    c |= np.where(rng.random((S, V)) < 0.02, 0x8000, 0).astype(np.uint16)
    path = rng.integers(-1, V, (B, R, P) if tree else (B, P)).astype(np.int32)
    if P > 1:
        path[..., 1] = path[..., 0]                    # the same id twice
    ids = rng.integers(-1, V, (B, nb)).astype(np.int32)
    if nb > 2:
        ids[:, 1] = ids[:, 0]
        ids[:, 2] = path.reshape(B, -1)[:, 0] if P else ids[:, 2]
    bias = rng.standard_normal((B, nb)).astype(np.float32) * 4
    on = rng.random((B, R, 32 * -(-V // 32))) < allowed
    on[:, 0, :V] |= rng.random((B, V)) < 0.9
    mask = np.packbits(on, axis=-1, bitorder="little").view(np.int32)
    f = lambda lo, hi: rng.uniform(lo, hi, B).astype(np.float32)   # noqa: E731
    return dict(logits=z, counts=c, slots=rng.permutation(S)[:B].astype(np.int32), path=path, repetition=f(0.7, 1.5),
                frequency=f(-0.5, 1), presence=f(-0.5, 1), bias_ids=ids, bias=bias, mask=mask)


def _run(c, dtype, in_place=False, **kw):
    import sampling_gated_lora_b200 as U
    z = dev_tensor(c["logits"], dtype)
    o = lambda k, t: None if c.get(k) is None else dev_tensor(c[k], t)   # noqa: E731
    keep = z.clone()
    out = U.logits_process(z, out=z if in_place else None, counts=None if c.get("counts") is None else _i16(c["counts"]),
                           slots=o("slots", "i32"), draft=o("path", "i32"), repetition=o("repetition", "f32"),
                           frequency=o("frequency", "f32"), presence=o("presence", "f32"), bias_ids=o("bias_ids", "i32"),
                           bias=o("bias", "f32"), mask=o("mask", "i32"), **kw)
    if not in_place:
        assert bool((z.view(-1) == keep.view(-1)).logical_or(z.view(-1).isnan()).all())
    return host_f64(out)


def _check(c, dtype, **kw):
    c = dict(c)
    if dtype == "bf16":
        c["logits"] = W.bf16_round(c["logits"])
        z = W.bf16_to_f64(c["logits"])
    else:
        c["logits"] = z = c["logits"].astype(np.float32)
    ref = L.process(z, **{k: v for k, v in c.items() if k != "logits"})
    got = _run(c, dtype, **kw)
    np.testing.assert_array_equal(np.isfinite(got), np.isfinite(ref))
    np.testing.assert_array_equal(got[~np.isfinite(ref)], ref[~np.isfinite(ref)])
    f = np.isfinite(ref)
    nb = 0 if c.get("bias") is None else c["bias"].shape[1]
    n = 6 + (int((c["counts"] & 0x7FFF).max()) if c.get("counts") is not None else 0)
    size = 1.5 * np.abs(z) + n + (np.abs(c["bias"]).sum(1)[:, None, None] if nb else 0)   # every term on the way
    tol = (5 + nb) * 2.0 ** -24 * size + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(np.where(f, ref, 0))
    assert np.all(np.abs(got[f] - ref[f]) <= tol[f])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,R,V,P,nb,tree", [
    (1, 1, 2, 0, 0, False), (1, 2, 31, 1, 1, False), (2, 9, 1000, 8, 3, False), (3, 5, 1001, 4, 7, True),
    (1, 3, 4099, 2, 300, False), (2, 2, 8192, 1, 1024, False), (1, 2, 8200, 64, 5, True), (2, 3, 151936, 2, 64, False),
    (1, 2, 151935, 1, 9, True), (1, 1, 196608, 1, 2, True)])
def test_rules_match_the_oracle(B, R, V, P, nb, tree, dtype):
    c = _case(B, R, V, P, nb, tree, seed=V + P)
    if P == 0:
        c["path"] = None
    if nb == 0:
        c["bias_ids"] = c["bias"] = None
    _check(c, dtype)
    _check(c, dtype, in_place=True)


@pytest.mark.parametrize("on", ["counts", "path", "bias", "mask", "none"])
def test_each_rule_alone(on):
    c = _case(2, 4, 1000, 3, 5, False, seed=11)
    if on != "counts":
        c["counts"] = c["slots"] = None
    if on not in ("counts", "path"):
        c["repetition"] = c["frequency"] = c["presence"] = None
    if on != "path":
        c["path"] = None
    if on != "bias":
        c["bias_ids"] = c["bias"] = None
    if on != "mask":
        c["mask"] = None
    _check(c, "f32")
    _check(c, "bf16", in_place=True)


@pytest.mark.parametrize("V", [1000, 1001])
def test_masked_places_hide_what_is_there_and_empty_rows_are_reported(V):
    import torch
    import sampling_gated_lora_b200 as U
    c = _case(1, 3, V, 2, 4, False, seed=V, allowed=0.5)
    on = np.unpackbits(c["mask"].view(np.uint8).reshape(1, 3, -1), axis=-1, bitorder="little")
    on[0, 1] = 0
    on[0, 1, V:] = 1                       # bits past the vocabulary allow nothing
    c["mask"] = np.packbits(on, axis=-1, bitorder="little").view(np.int32)
    z = c["logits"]
    z[0, 0][on[0, 0, :V] == 0] = np.nan
    z[0, 2][on[0, 2, :V] == 0] = np.inf
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run({**c, "logits": z}, "f32", dev_status=st)
    assert np.isneginf(got[0, 1]).all() and np.isneginf(got[0][on[0, :, :V] == 0]).all()
    assert np.isfinite(got[0, 0][on[0, 0, :V] != 0]).all() and np.isfinite(got[0, 2][on[0, 2, :V] != 0]).all()
    assert int(st) == U.DEV_NO_TOKEN and U.device_status() == U.DEV_NO_TOKEN


def test_values_that_are_not_finite_and_bad_ids():
    import torch
    import sampling_gated_lora_b200 as U
    c = _case(2, 2, 1000, 2, 3, False, seed=5)
    c["mask"] = None
    c["logits"][0, 0, :4] = [np.nan, np.inf, -np.inf, 0.0]
    c["counts"][:, :4] = 0x8001
    c["path"][0, 0], c["bias_ids"][1, 0], c["slots"][1] = 1000, -5, 77
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = L.process(c["logits"].astype(np.float32), **{k: v for k, v in c.items() if k != "logits"})
    got = _run(c, "f32", dev_status=st)
    np.testing.assert_allclose(got, ref, rtol=1e-5, atol=1e-5, equal_nan=True)
    assert int(st) == U.DEV_BAD_INDEX
    U.device_status()


def test_graph_replay_in_place_on_another_stream():
    import torch
    import sampling_gated_lora_b200 as U
    c = _case(2, 3, 1000, 2, 4, False, seed=8)
    z = dev_tensor(c["logits"], "f32")
    a = dict(counts=_i16(c["counts"]), slots=dev_tensor(c["slots"], "i32"), draft=dev_tensor(c["path"], "i32"),
             repetition=dev_tensor(c["repetition"], "f32"), mask=dev_tensor(c["mask"], "i32"))
    want = U.logits_process(z, **a)
    buf = z.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            U.logits_process(buf, out=buf, **a)
        for _ in range(2):
            buf.copy_(z)
            g.replay()
            assert torch.equal(buf, want)
