"""Cases of the 16-bit operators: the linear with its epilogue, the decode
layer with bf16 experts and the grouped expert FFN with bf16 experts.

`run` computes them in their plain form (elementary torch operations in fp32),
or, with `own` set, through quantized_moe_route_b200.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}

# The layer's shape is the benchmark's (hidden 2048, width 512, 256 experts, 8 a
# token), the tiny one the smallest that the tests use; linear sizes are
# multiples of that shape or generic odd ones.
H, F, E, K8 = 2048, 512, 256, 8


def _linear(name, T, N, K, dtype="bf16", act="none", gated=False, bias=False, residual=False, out32=False, pad=0):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "dtype": dtype, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "out32": out32, "pad": pad}


def _decode(name, T, E, k, H, F, shared="none", residual=False, router=True):
    return {"name": name, "op": "decode", "T": T, "E": E, "k": k, "H": H, "F": F, "shared": shared,
            "residual": residual, "router": router}


def _grouped(name, T, E, k, H, F, zipf):
    return {"name": name, "op": "grouped", "T": T, "E": E, "k": k, "H": H, "F": F, "zipf": zipf}


def listed():
    return [
        # one token's projection back onto the residual stream
        _linear("linear one token", 1, H, H, residual=True),
        # a decode batch's wide projection, odd sizes, rows of a wider buffer
        _linear("linear 13 tokens ragged", 13, 4099, 1000, "f16", "gelu", bias=True, pad=24),
        # the dense SwiGLU half of a shared expert for a short prompt
        _linear("linear gated 160 tokens", 160, F, H, act="silu", gated=True),
        # scores in fp32 over an odd vocabulary for a few hundred positions
        _linear("linear 333 tokens fp32 out", 333, 5001, H, bias=True, out32=True),
        # a long prompt's largest projection: the tensor-bound end
        _linear("linear 8192 tokens", 8192, 4 * H, H, act="gelu_tanh", bias=True, residual=True),
        # the tiny layer, logits given: latency only
        _decode("decode tiny 3 tokens", 3, 8, 2, 128, 64, router=False),
        # the benchmark's layer, one token a step: a serving step's unit
        _decode("decode one token", 1, E, K8, H, F),
        # a small batch with the sigmoid-gated shared expert and the residual
        _decode("decode 4 tokens shared", 4, E, K8, H, F, "gated", True),
        # the largest decode batch
        _decode("decode 16 tokens", 16, E, K8, H, F, "one"),
        # a short ragged prompt on a small layer
        _grouped("grouped 37 tokens small", 37, 8, 2, 256, 192, 0.0),
        # a prompt whose rows spread thinly over all experts: weight bound
        _grouped("grouped 100 tokens", 100, E, K8, H, F, 0.0),
        # the benchmark's prompt, expert loads skewed: tensor bound
        _grouped("grouped 2048 tokens skewed", 2048, E, K8, H, F, 1.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "decode", "grouped"))
    if op == "linear":
        c = _linear("", _log(rng, 1, 8192), _log(rng, 16, 8192), _log(rng, 64, 4096), rng.choice(("bf16", "f16")),
                    rng.choice(("none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid")), rng.random() < 0.3,
                    rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3, rng.choice((0, 0, 8, 40)))
        # no more work than the largest listed product
        c["T"] = min(c["T"], 8192 * 4 * H * H // ((1 + c["gated"]) * c["N"] * c["K"]))
    elif op == "decode":
        e = _log(rng, 4, 256)
        c = _decode("", rng.randint(1, 16), e, rng.randint(1, min(e, 10)), 64 * _log(rng, 2, 32), 64 * _log(rng, 1, 12),
                    rng.choice(("none", "one", "gated")), rng.random() < 0.5, rng.random() < 0.7)
    else:
        e = _log(rng, 4, 256)
        c = _grouped("", _log(rng, 1, 2048), e, rng.randint(1, min(e, 8)), 64 * _log(rng, 2, 32),
                     64 * _log(rng, 1, 8), rng.choice((0.0, 0.0, 1.1)))
    del c["name"]
    return c


def _normal(gen, shape, sigma, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=gen)


def _group_counts(case, seed):
    """Rows of each expert when T tokens pick k of E by N(0, 1) scores with a Zipf bias over a seeded order."""
    gen = torch.Generator().manual_seed(seed)
    n = case["E"]
    rank = torch.randperm(n, generator=gen) + 1
    scores = torch.randn((case["T"], n), generator=gen) - case["zipf"] * torch.log(rank.float())
    return torch.bincount(torch.topk(scores, case["k"], dim=1).indices.reshape(-1), minlength=n)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "linear":
        dt, T, N, K, pad = DTYPES[case["dtype"]], case["T"], case["N"], case["K"], case["pad"]
        rows = 2 * N if case["gated"] else N
        ld = (K + 7) // 8 * 8 + pad  # rows start on 16-byte boundaries
        s["x"] = _normal(gen, (T, ld), 1.0, dt)[:, :K]
        s["w"] = _normal(gen, (rows, ld), K ** -0.5, dt)[:, :K]
        s["bias"] = _normal(gen, (rows,), 0.5, dt) if case["bias"] else None
        s["residual"] = _normal(gen, (T, N + pad), 1.0, dt)[:, :N] if case["residual"] else None
        s["y"] = torch.empty((T, N + pad), dtype=torch.float32 if case["out32"] else dt, device="cuda")[:, :N]
        return s
    n, h, f = case["E"] + (case.get("shared", "none") != "none"), case["H"], case["F"]
    bf = torch.bfloat16
    s["gate_up"] = _normal(gen, (n, 2 * f, h), 0.02, bf)
    s["down"] = _normal(gen, (n, h, f), 0.02, bf)
    if case["op"] == "decode":
        T, k = case["T"], case["k"]
        s["x"] = _normal(gen, (T, h), 1.0, bf)
        s["wr"] = _normal(gen, (case["E"], h), h ** -0.5, bf) if case["router"] else None
        s["logits"] = (torch.empty((T, case["E"]), device="cuda") if case["router"]
                       else _normal(gen, (T, case["E"]), 1.0, torch.float32))
        s["gate"] = _normal(gen, (h,), h ** -0.5, bf) if case["shared"] == "gated" else None
        s["residual"] = _normal(gen, (T, h), 1.0, bf) if case["residual"] else None
        s["y"] = torch.empty((T, h), dtype=bf, device="cuda")
        s["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, k), device="cuda")
        return s
    offsets = torch.zeros(n + 1, dtype=torch.int32)
    offsets[1:] = torch.cumsum(_group_counts(case, seed), 0)
    rows = case["T"] * case["k"]
    s["offsets"] = offsets.cuda()
    s["x"] = _normal(gen, (rows, h), 1.0, bf)
    s["y"] = torch.empty((rows, h), dtype=bf, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _act(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return v


def _plain_linear(s):
    c, N = s["case"], s["case"]["N"]
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _act(v[:, :N], c["act"]) * v[:, N:] if c["gated"] else _act(v, c["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(s["y"].dtype)


def _plain_ffn(x, gate_up, down):
    """x [B][n][H] through gate_up [B][2F][H] and down [B][H][F], all fp32."""
    gu = torch.bmm(x, gate_up.transpose(1, 2))
    f = gu.shape[2] // 2
    return torch.bmm(_act(gu[..., :f], "silu") * gu[..., f:], down.transpose(1, 2))


def _plain_decode(s):
    c, x = s["case"], s["x"].float()
    T, k, n = c["T"], c["k"], c["E"]
    logits = x @ s["wr"].float().t() if c["router"] else s["logits"]
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: the lower id first
    top, idx = top[:, :k], idx[:, :k]
    e = torch.exp(top - top[:, :1])
    w = e / e.sum(1, keepdim=True)
    flat = idx.reshape(-1)
    rows = _plain_ffn(x.repeat_interleave(k, 0).unsqueeze(1), s["gate_up"][flat].float(), s["down"][flat].float())
    y = (rows.view(T, k, -1) * w.unsqueeze(2)).sum(1)
    if c["shared"] != "none":
        r = _plain_ffn(x.unsqueeze(0), s["gate_up"][n:].float(), s["down"][n:].float())[0]
        y = y + (_act(x @ s["gate"].float(), "sigmoid").unsqueeze(1) * r if s["gate"] is not None else r)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16), idx.to(torch.int32), w, logits


def _plain_grouped(s):
    x, off = s["x"], s["offsets"].long()
    rows, n = x.shape[0], off.numel() - 1
    r = torch.arange(rows, device="cuda")
    e = torch.searchsorted(off[1:], r, right=True)
    at = r - off[e]
    xp = torch.zeros((n, int((off[1:] - off[:-1]).max()), x.shape[1]), device="cuda")  # every expert's rows, padded
    xp[e, at] = x.float()
    return _plain_ffn(xp, s["gate_up"].float(), s["down"].float())[e, at].to(torch.bfloat16)


# ------------------------------------------------------------------ the framework's calls
def _workspace(s, need):
    """A call's workspace, kept with the plan like a user's program keeps it."""
    if "ws" not in s:
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    import quantized_moe_route_b200 as moe
    c = s["case"]
    if c["op"] == "linear":
        act = getattr(moe, "MOE_ACT_" + c["act"].upper())
        moe.moe_linear(s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"], act=act, gated=c["gated"])
        return s["y"]
    n, h, f = s["gate_up"].shape[0], c["H"], c["F"]
    if "layer" not in s:
        s["layer"] = moe.make_bf16_layer(n, h, f, s["gate_up"], s["down"])
    if c["op"] == "decode":
        shared = int(c["shared"] != "none")
        ws = _workspace(s, moe.moe_decode_layer_bf16_workspace_bytes(c["T"], c["k"], shared, n, h, f))
        moe.moe_decode_layer_bf16(s["layer"], s["x"], c["k"], s["y"], ws, wr=s["wr"], logits=s["logits"],
                                  shared=shared, shared_gate=s["gate"], residual=s["residual"], idx=s["idx"],
                                  w=s["w"])
        return s["y"], s["idx"], s["w"], s["logits"]
    ws = _workspace(s, moe.moe_prefill_bf16_workspace_bytes(s["x"].shape[0], f))
    moe.moe_ffn_grouped_prefill_bf16(s["layer"], s["x"], s["offsets"], s["y"], ws)
    return s["y"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_linear(state) if op == "linear" else _plain_decode(state) if op == "decode" else _plain_grouped(state)


def work(case):
    T = case["T"]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        rows = 2 * N if case["gated"] else N
        out = T * N * (4 if case["out32"] else 2)
        return {"bytes": 2 * (T * K + rows * K + case["bias"] * rows + case["residual"] * T * N) + out,
                "flops": 2 * T * rows * K}
    n, k, h, f = case["E"], case["k"], case["H"], case["F"]
    if case["op"] == "decode":
        shared = case["shared"] != "none"
        touched = n * (1 - (1 - k / n) ** T) + shared  # the expected number of different experts
        rows = T * (k + shared)
        small = 2 * T * h * (2 + case["residual"]) + 8 * T * k + 4 * T * n + 2 * h * (case["shared"] == "gated")
        return {"bytes": int(touched * 6 * h * f) + small + case["router"] * 2 * n * h,
                "flops": rows * 6 * h * f + case["router"] * 2 * T * n * h}
    counts = _group_counts(case, 1)
    rows = T * k
    return {"bytes": int((counts > 0).sum()) * 6 * h * f + 4 * rows * h + 4 * (n + 1), "flops": rows * 6 * h * f}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_act(v, name):
    one = torch.ones((), dtype=torch.float64, device=v.device)
    if name == "silu":
        return v * torch.special.expit(v)
    if name == "sigmoid":
        return torch.special.expit(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        # (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
        return v * torch.special.expit(2 * torch.sqrt(2 * one / math.pi) * (v + 0.044715 * v ** 3))
    if name == "relu":
        return torch.clamp(v, min=0)
    return v


def _exact_expert(s, e, x):
    """Expert e's FFN of the rows x (64 bits)."""
    w, d = s["gate_up"][e].double(), s["down"][e].double()
    f = d.shape[1]
    return (_exact_act(x @ w[:f].T, "silu") * (x @ w[f:].T)) @ d.T


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "linear":
        N = case["N"]
        out = torch.empty((case["T"], N), dtype=torch.float64, device="cuda")
        w = s["w"].double()
        b = s["bias"].double() if case["bias"] else torch.zeros(w.shape[0], dtype=torch.float64, device="cuda")
        if case["gated"]:
            out[:] = _exact_act(x @ w[:N].T + b[:N], case["act"]) * (x @ w[N:].T + b[N:])
        else:
            out[:] = _exact_act(x @ w.T + b, case["act"])
        if case["residual"]:
            out += s["residual"].double()
        return out
    if case["op"] == "decode":
        T, k = case["T"], case["k"]
        logits = torch.stack([s["wr"].double() @ x[t] for t in range(T)]) if case["router"] else s["logits"].double()
        y, w_out = torch.zeros_like(x), torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for t, row in enumerate(logits.tolist()):
            pick = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
            w_out[t] = torch.softmax(logits[t, pick], 0)
            for j, e in enumerate(pick):
                y[t] += w_out[t, j] * _exact_expert(s, e, x[t:t + 1])[0]
        if case["shared"] != "none":
            r = _exact_expert(s, case["E"], x)
            y += r * torch.special.expit(x @ s["gate"].double()).unsqueeze(1) if case["shared"] == "gated" else r
        if case["residual"]:
            y += s["residual"].double()
        return y, None, w_out, logits
    off = s["offsets"].tolist()
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        if off[e + 1] > off[e]:
            y[off[e]:off[e + 1]] = _exact_expert(s, e, x[off[e]:off[e + 1]])
    return y
