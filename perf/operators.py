"""The decode and training operators on 8-bit weights and on logits, as cases to measure.

Each case is one call of one operator: `prepare` makes what a program holds
before the call, `run` makes the call (`own` true: this package's entry
points; `own` false: the same mathematics in elementary torch operations in
32 bits), `exact` restates it in 64 bits from the definition.

  quantize  fp8_quantize: e4m3 codes and a float scale for each 1 x 128 or 128 x 128 block
  linear    gated_lora_linear_fp8: y = x W^T + s g (x A^T) Bl^T, W and x in e4m3 blocks of 128
  grad      gated_lora_input_grad_fp8: dx = dy W + s g (dy Bl) A, W and dy in e4m3 blocks of 128
  counts    token_counts_add: which tokens a sequence holds, and how often it emitted each
  logits    logits_process: repetition, frequency and presence penalties, biases, grammar masks
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100   # smallest block maximum a scale is taken from


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the 9 token rows of one sequence's verified block (k = 8 and the anchor), before a projection
        dict(name="quantize_decode_rows", op="quantize", M=9, K=4096, block_rows=1),
        # an MLP weight matrix put into 8 bits when a checkpoint is loaded
        dict(name="quantize_mlp_weight", op="quantize", M=12288, K=4096, block_rows=128),
        # attention projection of one sequence's step: the latency of a single user
        dict(name="linear_decode_9", op="linear", M=9, K=4096, N=4096, r=128),
        # a small ragged stack (tests and tiny drafters): no size on the tile grid
        dict(name="linear_ragged_77", op="linear", M=77, K=1040, N=1000, r=24),
        # LM head of a step of 8 sequences (8 (2 * 8 + 1) rows)
        dict(name="linear_head_136", op="linear", M=136, K=4096, N=151936, r=128),
        # MLP down-projection of a step of 256 sequences: the largest step
        dict(name="linear_down_4352", op="linear", M=4352, K=12288, N=4096, r=128),
        # input gradient of a small ragged layer
        dict(name="grad_ragged_33", op="grad", M=33, K=1000, N=1040, r=24),
        # input gradient of the MLP up-projection on a clean + noisy training batch (64 sequences of 16)
        dict(name="grad_up_2048", op="grad", M=2048, K=4096, N=12288, r=128),
        # the tokens one verified step emitted, 256 sequences
        dict(name="counts_step_256", op="counts", B=256, T=9, V=151936, prompt=False),
        # prompts of 32 newly admitted sequences
        dict(name="counts_prompts", op="counts", B=32, T=8192, V=151936, prompt=True),
        # AR rows of one sequence's candidate tree (8 blocks of 4: at most 33 nodes), float logits
        dict(name="logits_tree_f32", op="logits", B=1, R=33, P=4, V=32000, nb=16, allowed=0.03, dtype="f32", tree=True),
        # AR rows of a step of 256 sequences (k = 8 and the bonus row), every rule on
        dict(name="logits_verify_256", op="logits", B=256, R=9, P=8, V=151936, nb=64, allowed=0.05, dtype="bf16", tree=False),
    ]


def _log(rng, lo, hi, step=1):
    return max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "grad", "counts", "logits", "logits"])
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 12288), K=_log(rng, 64, 4096, 8), block_rows=rng.choice([1, 128]))
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 4352), K=_log(rng, 128, 12288, 16), N=_log(rng, 64, 4096, 8), r=rng.choice([0, 8, 24, 64, 128, 200]))
    if op == "grad":
        return dict(op=op, M=_log(rng, 1, 2048), K=_log(rng, 64, 4096, 8), N=_log(rng, 128, 12288, 16), r=rng.choice([0, 8, 24, 64, 128, 200]))
    if op == "counts":
        prompt = rng.random() < 0.5
        return dict(op=op, B=_log(rng, 1, 32 if prompt else 256), T=_log(rng, 1, 8192 if prompt else 33), V=_log(rng, 1000, 151936), prompt=prompt)
    tree = rng.random() < 0.3
    R = rng.randint(2, 33)
    return dict(op=op, B=_log(rng, 1, 32), R=R, P=rng.randint(1, 8) if tree else R - 1, V=_log(rng, 1000, 151936), nb=rng.choice([0, 1, 30, 300]),
                allowed=rng.choice([0.001, 0.05, 0.5, 1.0]), dtype=rng.choice(["bf16", "f32"]), tree=tree)


def _blocks(n, b=128):
    return -(-n // b)


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["M"] * c["K"]
        return {"bytes": 3 * n + 4 * _blocks(c["M"], c["block_rows"]) * _blocks(c["K"]), "flops": 3 * n}
    if c["op"] in ("linear", "grad"):
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        return {"bytes": 2 * M * (K + N) + N * K + 4 * _blocks(N) * _blocks(K) + 2 * r * (K + N) + M, "flops": 2 * M * N * K + 2 * M * r * (K + N)}
    if c["op"] == "counts":
        n = c["B"] * c["T"]
        return {"bytes": 4 * n + 4 * n + 8 * c["B"], "flops": n}   # tokens in; a 16-bit word read and written for each
    esz = 2 if c["dtype"] == "bf16" else 4
    rows, V = c["B"] * c["R"], c["V"]
    return {"bytes": 2 * rows * V * esz + 2 * c["B"] * V + 4 * rows * _blocks(V, 32) + 8 * c["B"] * c["nb"] + 4 * c["B"] * c["P"] * (c["R"] if c["tree"] else 1), "flops": 6 * rows * V}


# ---------------------------------------------------------------- inputs

def _weights_fp8(n_out, n_in, g):
    """A weight matrix in blocks of 128 x 128, as a checkpoint in 8 bits holds it: codes and float scales."""
    codes = torch.empty(n_out, n_in, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(_blocks(n_out), _blocks(n_in), device=DEV)
    step = 128 * 64
    for i in range(0, n_out, step):
        w = torch.randn(min(step, n_out - i), n_in, generator=g, device=DEV) * n_in ** -0.5
        codes[i:i + step], scales[i // 128:i // 128 + _blocks(w.shape[0])] = _quantize_plain(w, 128)
    return codes, scales


def _activations(M, K, g):
    """Normal activations with a few large channels, as hidden states have them."""
    x = torch.randn(M, K, generator=g, device=DEV)
    return (x * (1 + 15 * (torch.rand(K, generator=g, device=DEV) < 0.01))).bfloat16()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV)   # noqa: E731
    if c["op"] == "quantize":
        c["x"] = _activations(c["M"], c["K"], g) if c["block_rows"] == 1 else (rn(c["M"], c["K"]) * c["K"] ** -0.5).bfloat16()
    elif c["op"] in ("linear", "grad"):
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        if c["op"] == "linear":
            c["x"] = _activations(M, K, g)
            c["Wq"], c["Ws"] = _weights_fp8(N, K, g)
        else:   # the weight laid out once for its input gradient: transposed codes and scales
            c["dy"] = (rn(M, N) * 1e-2).bfloat16()
            c["Wqt"], c["Wst"] = _weights_fp8(K, N, g)
        c["A"] = (rn(r, K) * K ** -0.5).bfloat16() if r else None
        c["Bl"] = (rn(N, r) * 0.1).bfloat16() if r else None
        c["gate"] = (torch.rand(M, generator=g, device=DEV) < 0.5).to(torch.uint8)
        c["scale"] = 0.75
    elif c["op"] == "counts":
        B, T, V = c["B"], c["T"], c["V"]
        S = B + 3
        c["table"] = torch.where(torch.rand(S + 1, V, generator=g, device=DEV) < 0.01, 3, 0).to(torch.int16)   # one row more than the slots
        c["slots"] = torch.randperm(S, generator=g, device=DEV)[:B].to(torch.int32)
        c["tokens"] = (torch.rand(B, T, generator=g, device=DEV) ** 3 * V).to(torch.int32).clamp(max=V - 1)   # some ids far more often than others
        c["lens"] = ri(0, T + 1, B).to(torch.int32)
    else:
        B, R, V, P = c["B"], c["R"], c["V"], c["P"]
        z = rn(B * R, V) * 3.0
        peak = torch.rand(B * R, generator=g, device=DEV) < 0.05
        z[torch.arange(B * R, device=DEV), ri(0, V, B * R)] += 12.0 * peak
        c["logits"] = z.view(B, R, V).to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        S = B + 2
        u = torch.rand(S, V, generator=g, device=DEV)
        c["counts"] = torch.where(u < 0.002, 1 + (u * 1500).to(torch.int32), 0).add_(torch.where((u > 0.001) & (u < 0.01), -32768, 0)).to(torch.int16)
        c["slots"] = torch.randperm(S, generator=g, device=DEV)[:B].to(torch.int32)
        shape = (B, R, P) if c["tree"] else (B, P)
        c["draft"] = (torch.rand(shape, generator=g, device=DEV) ** 2 * V).to(torch.int32).clamp(max=V - 1)
        if c["tree"]:   # a node's path is as long as it is deep
            c["draft"] = torch.where(torch.arange(P, device=DEV) < ri(0, P + 1, B, R, 1), c["draft"], -1).to(torch.int32)
        c["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=DEV)
        c["frequency"] = 0.5 * torch.rand(B, generator=g, device=DEV)
        c["presence"] = 0.5 * torch.rand(B, generator=g, device=DEV)
        c["bias_ids"] = ri(0, V, B, c["nb"]).to(torch.int32) if c["nb"] else None
        c["bias"] = rn(B, c["nb"]) * 5 if c["nb"] else None
        c["mask"] = torch.empty(B, R, _blocks(V, 32), dtype=torch.int32, device=DEV)
        bit = torch.ones(32, dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
        for b in range(B):   # half of the sequences follow a grammar
            share = c["allowed"] if b % 2 == 0 else 1.0
            on = torch.rand(R, c["mask"].shape[2], 32, generator=g, device=DEV) < share
            c["mask"][b] = (on * bit).sum(-1).to(torch.int32)
    return c


# ---------------------------------------------------------------- plain forms

def _pad(x, rows, cols):
    M, K = x.shape
    return torch.nn.functional.pad(x, (0, _blocks(K, cols) * cols - K, 0, _blocks(M, rows) * rows - M))


def _quantize_plain(x, block_rows):
    """(codes, scales): scale = max |x| / 448 of the block, codes = e4m3(x * (448 / max |x|))."""
    M, K = x.shape
    p = _pad(x.float(), block_rows, 128)
    b = p.view(p.shape[0] // block_rows, block_rows, p.shape[1] // 128, 128)
    top = torch.full((), E4M3_MAX, device=x.device)
    amax = b.abs().amax(dim=(1, 3)).clamp_min(AMAX_FLOOR)
    codes = (b * (top / amax)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(p.shape)[:M, :K].contiguous(), amax / top


def _values(codes, scales, block_rows, dtype=torch.float32):
    M, K = codes.shape
    p = _pad(codes.to(dtype), block_rows, 128)
    b = p.view(scales.shape[0], block_rows, scales.shape[1], 128)
    return (b * scales.to(dtype)[:, None, :, None]).view(p.shape)[:M, :K]


def _product_plain(x, Wq, Ws, A, Bl, gate, scale):
    """x W^T + scale gate (x A^T) Bl^T with x and W held in e4m3 blocks; the adapter reads x itself."""
    y = _values(*_quantize_plain(x, 1), 1) @ _values(Wq, Ws, 128).T
    if A is not None:
        t = (scale * gate.float()[:, None] * (x.float() @ A.float().T)).bfloat16().float()   # the framework rounds t
        y = y + t @ Bl.float().T
    return y.bfloat16()


def _counts_plain(st):
    table, tok = st["table"], st["tokens"].long()
    B, T = tok.shape
    at = torch.arange(T, device=tok.device)
    valid = at < st["lens"][:, None]
    slot = torch.where(valid, st["slots"].long()[:, None], table.shape[0] - 1)   # what is not counted goes to the spare row
    old = table[slot, tok].int()
    if st["prompt"]:
        new = old | -32768
    else:
        times = ((tok[:, :, None] == tok[:, None, :]) & valid[:, None, :]).sum(-1)
        new = ((old & 0x7FFF) + times).clamp(max=0x7FFF) | (old & -32768)
    table[slot, tok] = new.to(torch.int16)
    table[-1] = 0
    return table[:-1]


def _logits_plain(st, dtype=torch.float32):
    z = st["logits"].to(dtype)
    B, R, V = z.shape
    word = st["counts"][st["slots"].long()].int()
    n = (word & 0x7FFF)[:, None, :].expand(B, R, V).to(torch.int32, copy=True)
    d = st["draft"]
    if d.dim() == 2:   # row j of a block follows its first j drafted tokens
        d = torch.where(torch.arange(d.shape[1], device=d.device) < torch.arange(R, device=d.device)[:, None], d[:, None, :], -1)
    n.scatter_add_(2, d.clamp_min(0).long(), (d >= 0).int())
    rho, freq, pres = (st[k].to(dtype)[:, None, None] for k in ("repetition", "frequency", "presence"))
    held = (n > 0) | (word < 0)[:, None, :]
    z = torch.where(held, torch.where(z > 0, z / rho, z * rho), z)
    z = z - freq * n - pres * (n > 0)
    if st["bias"] is not None:
        z = z.scatter_add(2, st["bias_ids"].long()[:, None, :].expand(B, R, -1), st["bias"].to(dtype)[:, None, :].expand(B, R, -1))
    on = (st["mask"][..., None] >> torch.arange(32, device=z.device, dtype=torch.int32)) & 1
    z = torch.where(on.view(B, R, -1)[..., :V] != 0, z, -math.inf)
    return z


# ---------------------------------------------------------------- one pass

def _kept(st, name, make):
    """A buffer that a program allocates at its first call and uses again."""
    if name not in st:
        st[name] = make()
    return st[name]


def _workspace(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=DEV)


def _run_own(st):
    import sampling_gated_lora_b200 as U
    op = st["op"]
    if op == "quantize":
        return U.fp8_quantize(st["x"], st["block_rows"])
    if op == "linear":
        x, Wq = st["x"], st["Wq"]
        ws = _kept(st, "workspace", lambda: _workspace(U.gated_lora_linear_fp8_workspace(x.shape[0], x.shape[1], Wq.shape[0], st["r"])))
        return U.gated_lora_linear_fp8(x, Wq, st["Ws"], st["A"], st["Bl"], st["gate"], st["scale"], workspace=ws)
    if op == "grad":
        dy, Wqt = st["dy"], st["Wqt"]
        ws = _kept(st, "workspace", lambda: _workspace(U.gated_lora_input_grad_fp8_workspace(dy.shape[0], Wqt.shape[0], Wqt.shape[1], st["r"])))
        return U.gated_lora_input_grad_fp8(dy, Wqt, st["Wst"], st["A"], st["Bl"], st["gate"], st["scale"], workspace=ws)
    if op == "counts":
        return U.token_counts_add(st["table"][:-1], st["tokens"], lens=st["lens"], slots=st["slots"], prompt=st["prompt"])
    return U.logits_process(st["logits"], counts=st["counts"], slots=st["slots"], draft=st["draft"], repetition=st["repetition"], frequency=st["frequency"],
                            presence=st["presence"], bias_ids=st["bias_ids"], bias=st["bias"], mask=st["mask"])


def run(state):
    st, op = state, state["op"]
    if own:
        return _run_own(st)
    if op == "quantize":
        return _quantize_plain(st["x"], st["block_rows"])   # codes as e4m3 numbers, and scales
    if op == "linear":
        return _product_plain(st["x"], st["Wq"], st["Ws"], st["A"], st["Bl"], st["gate"], st["scale"])
    if op == "grad":
        A, Bl = st["A"], st["Bl"]
        return _product_plain(st["dy"], st["Wqt"], st["Wst"], None if Bl is None else Bl.T, None if A is None else A.T, st["gate"], st["scale"])
    if op == "counts":
        return _counts_plain(st)
    return _logits_plain(st).to(st["logits"].dtype)


# ---------------------------------------------------------------- 64 bits

def _e4m3_64(v):
    """v rounded to the nearest e4m3 value (4 significant bits, steps of 2^-9 below 2^-6, ties to even), in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp_min(-9))
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _blockwise_64(x, rows):
    """x in blocks of rows x 128: (e4m3 values of x / scale, the scales), scale = max |x| / 448."""
    M, K = x.shape
    v, s = torch.empty(M, K, dtype=torch.float64, device=x.device), torch.empty(_blocks(M, rows), _blocks(K), dtype=torch.float64, device=x.device)
    for j in range(_blocks(K)):
        part = x[:, 128 * j:128 * j + 128].double()
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.nn.functional.pad(top, (0, _blocks(M, rows) * rows - M)).view(-1, rows).amax(1)
        s[:, j] = top.clamp_min(AMAX_FLOOR) / E4M3_MAX
        v[:, 128 * j:128 * j + 128] = _e4m3_64(part / s[:, j].repeat_interleave(rows)[:M, None])
    return v, s


def _product_64(x, Wq, Ws, A, Bl, gate, scale):
    v, s = _blockwise_64(x, 1)
    y = torch.zeros(x.shape[0], Wq.shape[0], dtype=torch.float64, device=x.device)
    for j in range(s.shape[1]):   # block by block along K: its own scales on both sides
        cut = slice(128 * j, 128 * j + 128)
        y += s[:, j:j + 1] * (v[:, cut] @ Wq[:, cut].to(torch.float32).double().T) * Ws[:, j].double().repeat_interleave(128)[:Wq.shape[0]]
    if A is not None:
        y += scale * gate.double()[:, None] * ((x.double() @ A.double().T) @ Bl.double().T)
    return y


def _logits_64(st):
    z = st["logits"]
    out = torch.empty(z.shape, dtype=torch.float64, device=z.device)
    B, R, V = z.shape
    for b in range(B):
        word = st["counts"][int(st["slots"][b])].to(torch.int64)
        emitted, prompt = word % 32768, word < 0
        rho, freq, pres = (float(st[k][b]) for k in ("repetition", "frequency", "presence"))
        extra = torch.zeros(V, dtype=torch.float64, device=z.device)
        if st["bias"] is not None:
            extra.index_add_(0, st["bias_ids"][b].long(), st["bias"][b].double())
        for i in range(R):
            path = st["draft"][b, i] if st["tree"] else st["draft"][b, :i]
            n = emitted + torch.bincount(path[path >= 0].long(), minlength=V)
            row = z[b, i].double()
            row = torch.where(prompt | (n > 0), torch.where(row > 0, row / rho, row * rho), row) - freq * n - pres * (n > 0).double() + extra
            bits = torch.from_numpy(np.unpackbits(st["mask"][b, i].cpu().numpy().view(np.uint8), bitorder="little")[:V].astype(bool)).to(z.device)
            row[~bits] = -math.inf
            out[b, i] = row
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "quantize":
        v, s = _blockwise_64(st["x"], st["block_rows"])
        return [v, s]
    if st["op"] == "linear":
        return _product_64(st["x"], st["Wq"], st["Ws"], st["A"], st["Bl"], st["gate"], st["scale"])
    if st["op"] == "grad":
        r = st["r"]
        return _product_64(st["dy"], st["Wqt"], st["Wst"], st["Bl"].T if r else None, st["A"].T if r else None, st["gate"], st["scale"])
    if st["op"] == "counts":
        return None   # whole numbers: the plain form is exact
    return _logits_64(st)
