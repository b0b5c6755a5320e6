"""GPU parity of the bf16-expert layer (moe_decode_layer_bf16,
moe_ffn_grouped_prefill_bf16) against the definition in 64 bits.

The grouped call rounds h to bf16, and its reference does so where the kernel
does; the decode layer keeps at least 16 significant bits of h, and its
reference keeps h as it is.  Tolerance per element of a row output:
  - h of the grouped call may round to the neighbouring bf16 value where its
    fp32 value is off by a hair: at most one bf16 step, 2^-7 |h|; h of the decode
    layer is off by at most 2^-16 |h|;
  - dh, the fp32 error of SiLU(g) u itself;
  - so a row is off by at most sum_f |Wd| (step |h| + dh), plus its fp32 sum, (2 F +
    2) 2^-23 sum |Wd||h|; the combine weighs rows by w (each off by 1e-6
    relative), and bf16 rounding adds 2^-8 |y|.
The relative L2 error is also held to rounding size: at most half a step, 2^-8.
"""
import math

import numpy as np
import pytest
import torch

import quantized_moe_route_b200 as moe
from moe_testlib import ffn_close

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normal(gen, shape, sigma):
    return torch.empty(shape, dtype=BF, device="cuda").normal_(0.0, sigma, generator=gen)


class Layer16:
    def __init__(self, seed, E, H, F, sigma=0.02):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.H, self.F = E, H, F
        self.gu, self.dn = normal(gen, (E, 2 * F, H), sigma), normal(gen, (E, H, F), sigma)
        self.desc = moe.make_bf16_layer(E, H, F, self.gu, self.dn)

    def rows(self, e, x):
        """Expert e's rows of x [n][H] and their tolerance, in 64 bits: from h rounded to bf16, and as it is."""
        H, F = self.H, self.F
        x, w, d = x.double(), self.gu[e].double(), self.dn[e].double()
        g, u = x @ w[:F].t(), x @ w[F:].t()
        A = (H + 2) * 2.0 ** -23 * (x.abs() @ w.abs().t())
        s = g * torch.special.expit(g)
        h = s * u
        dh = (1.2 * A[:, :F] + 2.0 ** -19 * s.abs().clamp(min=0.25)) * (u.abs() + A[:, F:]) + s.abs() * A[:, F:]
        hb = h.float().to(BF).double()
        tol, tol16 = ((step * h.abs() + dh + (2 * F + 2) * 2.0 ** -23 * (h.abs() + dh)) @ d.abs().t()
                      for step in (2.0 ** -7, 2.0 ** -16))
        return (hb @ d.t(), tol, h, dh), (h @ d.t(), tol16)


def reference(layer, x, lg, k, shared, gate, residual):
    T, H = x.shape
    Er = layer.E - shared
    lg = lg.double()
    order = sorted_experts(lg)
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    w = torch.empty((T, k), dtype=torch.float64)
    for t in range(T):
        pick = order[t][:k]
        w[t] = torch.softmax(lg[t, pick], 0).cpu()
        for j, e in enumerate(pick):
            r, tr = layer.rows(e, x[t:t + 1])[1]
            y[t] += w[t, j].item() * r[0]
            tol[t] += w[t, j].item() * (tr[0] + 2e-6 * r[0].abs())
    if shared:
        r, tr = layer.rows(Er, x)[1]
        if gate is not None:
            z = x.double() @ gate.double()
            dz = (H + 2) * 2.0 ** -23 * (x.double().abs() @ gate.double().abs())
            s = torch.special.expit(z).unsqueeze(1)
            tr = s * tr + (0.25 * dz.unsqueeze(1) + 2.0 ** -19) * r.abs()
            r = s * r
        y, tol = y + r, tol + tr
    if residual is not None:
        y = y + residual.double()
    tol = tol + 2.0 ** -8 * (y.abs() + tol) + 2.0 ** -22 * (residual.double().abs() if residual is not None else 0)
    return y, tol, order, w


def sorted_experts(lg):
    return [sorted(range(lg.shape[1]), key=lambda e, r=r: (-r[e], e)) for r in lg.tolist()]


def workspace(layer, T, k, shared):
    n = moe.moe_decode_layer_bf16_workspace_bytes(T, k, shared, layer.E, layer.H, layer.F)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def check_close(y, want, tol, what):
    err = (y.double() - want).abs()
    assert (err <= tol).all(), f"{what}: {(err - tol).max():.3e} past the bound"
    rel = (err.norm() / want.norm()).item()
    assert rel <= 2.0 ** -8, f"{what}: rel {rel:.2e}"


def run_decode(layer, x, k, shared=0, wr=None, lg=None, gate=None, residual=None, ws=None, y=None, stream=None):
    T = x.shape[0]
    y = torch.full((T, layer.H), 7.0, dtype=BF, device="cuda") if y is None else y
    idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    ws = workspace(layer, T, k, shared) if ws is None else ws
    out_lg = torch.full((T, layer.E - shared), float("nan"), device="cuda") if wr is not None else lg
    moe.moe_decode_layer_bf16(layer.desc, x, k, y, ws, wr=wr, logits=out_lg, shared=shared, shared_gate=gate,
                              residual=residual, idx=idx, w=w, stream=stream)
    return y, idx, w, out_lg


def check_decode(seed, T, E, k, H, F, shared="none", residual=False, router=True, x=None, lg=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = int(shared != "none")
    layer = Layer16(seed + 1, E + s, H, F)
    x = normal(gen, (T, H), 1.0) if x is None else x
    wr = normal(gen, (E, H), H ** -0.5) if router else None
    gate = normal(gen, (H,), H ** -0.5) if shared == "gated" else None
    res = normal(gen, (T, H), 1.0) if residual else None
    lg = None if router else (torch.randn((T, E), generator=gen, device="cuda") if lg is None else lg)
    y, idx, w, out_lg = run_decode(layer, x, k, s, wr, lg, gate, res)
    torch.cuda.synchronize()
    assert moe.moe_device_error() == 0
    if router:
        want_lg = x.double() @ wr.double().t()
        bound = (H + 2) * 2.0 ** -23 * (x.double().abs() @ wr.double().abs().t())
        assert ((out_lg.double() - want_lg).abs() <= bound).all()
    # the selection is exact on the logits that the call computed or was given
    want, tol, order, ww = reference(layer, x, out_lg, k, s, gate, res)
    assert idx.cpu().tolist() == [o[:k] for o in order]
    np.testing.assert_allclose(w.cpu().double().numpy(), ww.numpy(), rtol=1e-6, atol=1e-30)
    check_close(y, want, tol, "y")
    return layer, x, y


@pytest.mark.parametrize("T,E,k,H,F,shared,residual,router", [
    (1, 1, 1, 64, 64, "none", False, True), (1, 8, 2, 128, 64, "none", False, False),
    (4, 8, 2, 128, 64, "gated", True, True), (1, 256, 8, 2048, 512, "none", False, True),
    (2, 256, 8, 2048, 512, "one", True, False), (3, 5, 5, 192, 320, "gated", False, False),
    (5, 17, 3, 320, 128, "one", False, True), (7, 100, 10, 512, 192, "none", True, True),
    (8, 64, 8, 1024, 256, "gated", True, True), (9, 64, 8, 1024, 256, "none", False, True),
    (13, 30, 4, 832, 448, "one", True, True), (16, 256, 8, 2048, 512, "gated", True, True),
    (16, 64, 16, 256, 128, "none", False, True), (16, 64, 15, 256, 128, "one", False, False),
    (3, 1024, 8, 256, 128, "none", False, True), (2, 1023, 31, 128, 64, "gated", True, True),
    (6, 300, 32, 128, 64, "none", False, True), (1, 4, 2, 4096, 1536, "none", False, True),
    (2, 3, 1, 7168, 64, "one", True, True), (1, 2, 2, 64, 2048, "none", True, True),
    (16, 8, 8, 2048, 768, "gated", False, True)])
def test_decode_layer(T, E, k, H, F, shared, residual, router):
    check_decode(T * 1000 + E, T, E, k, H, F, shared, residual, router)


# several 512-input chunks to a down projection (the last one short), shared out over the warps; several strips a CTA
@pytest.mark.parametrize("T,E,k,H,F,shared", [
    (12, 16, 7, 2560, 1088, "none"), (16, 8, 3, 2432, 1408, "one"), (2, 64, 7, 64, 1472, "none"),
    (5, 8, 4, 4800, 576, "gated"), (1, 8, 2, 2496, 3968, "none"), (4, 16, 8, 512, 2560, "one")])
def test_decode_down_projection_of_many_chunks(T, E, k, H, F, shared):
    layer, x, y = check_decode(T * 77 + F, T, E, k, H, F, shared, True, False)
    lg = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(F), device="cuda")
    first = run_decode(layer, x, k, int(shared != "none"), lg=lg)[0]
    for _ in range(20):  # the chunks' sums meet in their order: the same bits
        assert torch.equal(run_decode(layer, x, k, int(shared != "none"), lg=lg)[0], first)


def test_decode_every_token_the_same_experts_and_ties():
    """All 16 tokens pick the same experts (every slot holds 16 tokens), from logits with equal values."""
    T, E, k, H, F = 16, 64, 8, 512, 256
    lg = torch.zeros((T, E), device="cuda")
    lg[:, 40:] = 1.0  # 24 equal best: the lower ids 40..47 win
    check_decode(71, T, E, k, H, F, router=False, lg=lg)
    lg = torch.randn((1, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).expand(T, E).contiguous()
    check_decode(72, T, E, k, H, F, "one", True, router=False, lg=lg)


def test_decode_masked_logits_and_large_logits():
    """Experts masked with -inf or the type's lowest value are not chosen while others remain."""
    T, E, k, H, F = 3, 40, 4, 128, 64
    lg = torch.randn((T, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    lg[0, 4:] = float("-inf")
    lg[1, 3:39] = torch.finfo(torch.float32).min
    lg[2] = lg[2] * 1e30
    check_decode(73, T, E, k, H, F, router=False, lg=lg)


def test_decode_exact_on_integers():
    """SiLU(g) = g in fp32 for g >= 32, so with integers every row is exact: one expert of weight 1 per token, y
    is the exact integer rounded once."""
    E, H, F, T = 4, 128, 64, 16
    gen = torch.Generator(device="cuda").manual_seed(8)
    gu = torch.zeros((E, 2 * F, H), dtype=BF, device="cuda")
    gu[:, :F, 0] = 32.0
    gu[:, F:, 1:] = torch.randint(-1, 2, (E, F, H - 1), generator=gen, device="cuda").to(BF) * (
        torch.rand((E, F, H - 1), generator=gen, device="cuda") < 0.05)
    dn = torch.randint(-3, 4, (E, H, F), generator=gen, device="cuda").to(BF)
    layer = Layer16.__new__(Layer16)
    layer.E, layer.H, layer.F, layer.gu, layer.dn = E, H, F, gu, dn
    layer.desc = moe.make_bf16_layer(E, H, F, gu, dn)
    x = torch.ones((T, H), dtype=BF, device="cuda")
    x[:, 1:] = torch.randint(-1, 2, (T, H - 1), generator=gen, device="cuda").to(BF)
    lg = torch.randn((T, E), generator=gen, device="cuda")
    y, idx, _, _ = run_decode(layer, x, 1, lg=lg)
    for t in range(T):
        e = int(lg[t].argmax())
        assert int(idx[t, 0]) == e
        u = x[t].double() @ gu[e, F:].double().t()
        assert u.abs().max() <= 255
        want = (32 * u) @ dn[e].double().t()
        assert torch.equal(y[t], want.float().to(BF))
    # the grouped call on the same rows: bf16 of the same integers
    order = torch.argsort(idx[:, 0].long(), stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(idx[:, 0].long(), minlength=E).cumsum(0)
    y2 = torch.empty((T, H), dtype=BF, device="cuda")
    ws2 = torch.empty(moe.moe_prefill_bf16_workspace_bytes(T, F), dtype=torch.uint8, device="cuda")
    moe.moe_ffn_grouped_prefill_bf16(layer.desc, x[order].contiguous(), offsets, y2, ws2)
    assert torch.equal(y2, y[order])


def test_decode_workspace_serves_calls_of_other_sizes():
    """One workspace, calls of changing T, k and router use: stale words of larger calls are never taken up."""
    layer = Layer16(80, 33, 256, 128)
    gen = torch.Generator(device="cuda").manual_seed(81)
    wr = normal(gen, (32, 256), 256 ** -0.5)
    ws = workspace(layer, 16, 8, 1)
    for i, (T, k, shared, router) in enumerate([(16, 8, 1, 1), (1, 2, 0, 0), (16, 8, 1, 1), (3, 8, 1, 0), (2, 1, 0, 1),
                                                (16, 4, 0, 1), (1, 8, 1, 1), (9, 8, 0, 0)]):
        E = layer.E - shared
        x = normal(gen, (T, 256), 1.0)
        w = torch.cat([wr, wr[:1]])[:E].contiguous() if router else None
        lg = None if router else torch.randn((T, E), generator=gen, device="cuda")
        y, idx, _, out_lg = run_decode(layer, x, k, shared, w, lg, ws=ws)
        torch.cuda.synchronize()
        assert moe.moe_device_error() == 0
        want, tol, order, _ = reference(layer, x, out_lg, k, shared, None, None)
        assert idx.cpu().tolist() == [o[:k] for o in order], i
        check_close(y, want, tol, f"call {i}")


def test_decode_residual_in_place_and_optional_outputs():
    layer = Layer16(85, 16, 256, 128)
    gen = torch.Generator(device="cuda").manual_seed(86)
    x, r, lg = normal(gen, (5, 256), 1.0), normal(gen, (5, 256), 1.0), torch.randn((5, 16), generator=gen, device="cuda")
    y1, _, _, _ = run_decode(layer, x, 4, lg=lg, residual=r)
    y2 = r.clone()
    moe.moe_decode_layer_bf16(layer.desc, x, 4, y2, workspace(layer, 5, 4, 0), logits=lg, residual=y2)
    assert torch.equal(y1, y2)
    wr = normal(gen, (16, 256), 256 ** -0.5)
    y3, idx, w, out_lg = run_decode(layer, x, 4, wr=wr)
    y4 = torch.empty_like(y3)
    moe.moe_decode_layer_bf16(layer.desc, x, 4, y4, workspace(layer, 5, 4, 0), wr=wr)
    assert torch.equal(y3, y4)
    # the layer given the logits that it computed: the same bits
    y5, idx5, w5, _ = run_decode(layer, x, 4, lg=out_lg)
    assert torch.equal(y3, y5) and torch.equal(idx, idx5) and torch.equal(w, w5)


def test_decode_captured_replays_and_streams():
    layer = Layer16(90, 65, 512, 256)
    gen = torch.Generator(device="cuda").manual_seed(91)
    T, k = 4, 6
    wr, gate = normal(gen, (64, 512), 512 ** -0.5), normal(gen, (512,), 512 ** -0.5)
    x, r = normal(gen, (T, 512), 1.0), normal(gen, (T, 512), 1.0)
    y = torch.empty((T, 512), dtype=BF, device="cuda")
    ws = workspace(layer, T, k, 1)
    call = lambda: moe.moe_decode_layer_bf16(layer.desc, x, k, y, ws, wr=wr, shared=1, shared_gate=gate, residual=r)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()  # two calls on one workspace in one graph, in order
    for i in range(4):
        x.copy_(normal(gen, (T, 512), 1.0))
        r.copy_(normal(gen, (T, 512), 1.0))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y_ref, _, _, _ = run_decode(layer, x, k, 1, wr=wr, gate=gate, residual=r)
        assert torch.equal(got, y_ref), i
    assert moe.moe_device_error() == 0
    # another stream, and two streams at once with a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(y) for _ in range(2)]
    wss = [workspace(layer, T, k, 1) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, w_ in zip(streams, outs, wss):
            moe.moe_decode_layer_bf16(layer.desc, x, k, o, w_, wr=wr, shared=1, shared_gate=gate, residual=r, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], y_ref) and torch.equal(outs[1], y_ref)
    assert moe.moe_device_error() == 0


@pytest.mark.parametrize("T", [1, 3, 11])
def test_decode_wait_that_runs_out_is_reported_and_leaves_the_gpu_usable(T):
    """Phase A publishes no h: every wait of phase B gives up within its bound, the call ends, the error word names
    the wait, and the next call on a cleared workspace is right."""
    layer = Layer16(95, 16, 512, 256)
    gen = torch.Generator(device="cuda").manual_seed(96)
    x, lg = normal(gen, (T, 512), 1.0), torch.randn((T, 16), generator=gen, device="cuda")
    ws, y = workspace(layer, T, 4, 0), torch.empty((T, 512), dtype=BF, device="cuda")
    assert moe.moe_device_error() == 0
    moe.moe_debug_starve_decode_bf16(layer.desc, x, lg, 4, y, ws, 500)
    torch.cuda.synchronize()
    assert moe.moe_device_error() == moe.MOE_DEVERR_DECODE_H_WAIT
    assert moe.moe_device_error() == 0
    ws.zero_()
    y, _, _, _ = run_decode(layer, x, 4, lg=lg, ws=ws)
    want, tol, _, _ = reference(layer, x, lg, 4, 0, None, None)
    check_close(y, want, tol, "the call after")
    assert moe.moe_device_error() == 0


@pytest.mark.parametrize("T", [1, 4, 7])
@pytest.mark.parametrize("H", [128, 192, 1088])
def test_decode_infinite_input_gives_infinite_output(T, H):
    """With weights above zero an infinite input makes every sum of its token +inf, wherever it lies, and no other
    token's anything else (a product of an infinity with padding would make them NaN)."""
    layer = Layer16(97, 8, H, 128)
    layer.gu.abs_().add_(0.01)
    layer.dn.abs_().add_(0.01)
    gen = torch.Generator(device="cuda").manual_seed(98)
    lg = torch.randn((T, 8), generator=gen, device="cuda")
    for at in sorted({0, 63, 64, H - 65, H - 1}):
        x = normal(gen, (T, H), 1.0).abs_()
        x[T - 1, at] = float("inf")
        y, _, _, _ = run_decode(layer, x, 2, lg=lg)
        assert torch.isinf(y[T - 1]).all() and (y[T - 1] > 0).all(), at
        assert torch.isfinite(y[: T - 1]).all(), at


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("ups, h", [((2.0**64, 0.0, 0.0), math.inf),
                                    ((2.0**63, 2.0**63 * (1 - 2.0**-8), 2.0**53), 2.0**128 * (1 - 2.0**-9 + 2.0**-11))])
def test_decode_h_at_the_end_of_the_range(T, ups, h):
    """An h beyond fp32 is inf on its way to the down projection, and one that fp32 holds but that bf16 would round to
    inf is finite.  One feature: silu(2^64) = 2^64, up the sum of three inputs' weights, down 2^-20."""
    H, F = 128, 64
    layer = Layer16(99, 4, H, F)
    layer.gu.zero_()
    layer.dn.zero_()
    layer.gu[:, 0, 0] = 1.0
    for i, u in enumerate(ups):
        layer.gu[:, F, 1 + i] = u
    layer.dn[:, :, 0] = 2.0**-20
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[:, 0] = 2.0**64
    x[:, 1:4] = 1.0
    y, _, _, _ = run_decode(layer, x, 1, lg=torch.zeros((T, 4), device="cuda"))
    assert torch.equal(y, torch.full_like(y, h * 2.0**-20))


# ------------------------------------------------------------------ grouped
def check_grouped(seed, counts, H, F, extra=0):
    E, rows = len(counts), sum(counts)
    layer = Layer16(seed, E, H, F)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = normal(gen, (rows + extra, H), 1.0)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    y = torch.full((rows + extra, H), 7.0, dtype=BF, device="cuda")
    n = moe.moe_prefill_bf16_workspace_bytes(rows + extra, F)
    ws = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_ffn_grouped_prefill_bf16(layer.desc, x, offsets, y, ws)
    torch.cuda.synchronize()
    assert moe.moe_device_error() == 0
    assert (y[rows:] == 7.0).all(), "rows of no expert were written"
    assert (ws[n:] == 0x5A).all()
    h = ws[:(rows + extra) * F * 2].view(BF).view(rows + extra, F)[:rows]
    at = 0
    for e, c in enumerate(counts):
        if c:
            want, tol, h64, dh = layer.rows(e, x[at:at + c])[0]
            herr = (h[at:at + c].double() - h64).abs()
            assert (herr <= 2.0 ** -8 * (h64.abs() + dh) + dh).all(), f"h of expert {e}"
            check_close(y[at:at + c], want, tol + 2.0 ** -8 * (want.abs() + tol), f"expert {e}")
        at += c


@pytest.mark.parametrize("counts,H,F,extra", [
    ([1], 64, 64, 0), ([3, 0, 5], 128, 64, 0), ([0, 0, 7, 0], 192, 192, 3), ([128, 127, 129, 1], 256, 128, 0),
    ([300, 0, 31, 257], 512, 320, 1), ([16] * 9, 2048, 512, 0), ([1] * 40, 320, 64, 0), ([513, 2, 0, 255], 64, 448, 130),
    ([0] * 7 + [260], 1088, 64, 0), ([700], 2048, 512, 0), ([0, 0, 0], 128, 64, 4), ([64, 65, 63, 200], 896, 576, 0)])
def test_grouped(counts, H, F, extra):
    if sum(counts) + extra:
        check_grouped(sum(counts) + H, counts, H, F, extra)


def test_grouped_at_the_expert_limit():
    rng = np.random.RandomState(3)
    counts = rng.poisson(0.6, 1024).tolist()
    check_grouped(99, counts, 128, 64)


def test_grouped_offsets_past_the_rows_are_clamped():
    """A table that claims more rows than the call has: the rows below still get their experts' outputs, nothing
    past them is written or read."""
    H, F, rows, pad = 128, 64, 100, 60
    layer = Layer16(101, 4, H, F)
    x = normal(torch.Generator(device="cuda").manual_seed(102), (rows + pad, H), 1.0)
    offsets = torch.tensor([0, 30, 60, 100, 160], dtype=torch.int32, device="cuda")
    y = torch.full((rows + pad, H), 7.0, dtype=BF, device="cuda")
    ws = torch.full((moe.moe_prefill_bf16_workspace_bytes(rows + pad, F),), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_ffn_grouped_prefill_bf16(layer.desc, x[:rows], offsets, y[:rows], ws)
    torch.cuda.synchronize()
    assert (y[rows:] == 7.0).all() and (ws[rows * F * 2:] == 0x5A).all()
    for e, (a, b) in enumerate([(0, 30), (30, 60), (60, 100)]):
        want, tol = layer.rows(e, x[a:b])[0][:2]
        check_close(y[a:b], want, tol + 2.0 ** -8 * (want.abs() + tol), f"expert {e}")


def test_grouped_captured_with_many_tiles():
    """Enough tiles for the counters (cleared in the graph): replays on new groups, and twice on the same."""
    E, H, F, rows = 160, 64, 256, 3000
    layer = Layer16(115, E, H, F, sigma=0.1)
    gen = torch.Generator(device="cuda").manual_seed(116)
    x, y = normal(gen, (rows, H), 1.0), torch.empty((rows, H), dtype=BF, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_prefill_bf16_workspace_bytes(rows, F), dtype=torch.uint8, device="cuda").fill_(0xFF)
    call = lambda: moe.moe_ffn_grouped_prefill_bf16(layer.desc, x, offsets, y, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    rng = np.random.RandomState(117)
    for i in range(3):
        p = rng.gamma(0.3, size=E) + 1e-9
        off = np.concatenate([[0], np.cumsum(rng.multinomial(rows, p / p.sum()))])
        offsets.copy_(torch.tensor(off, dtype=torch.int32))
        for _ in range(2):
            y.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert moe.moe_device_error() == 0
            for e in np.flatnonzero(np.diff(off)):
                a, b = off[e], off[e + 1]
                want, tol = layer.rows(int(e), x[a:b])[0][:2]
                assert ((y[a:b].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all(), (i, e)


def test_grouped_captured_follows_new_offsets():
    layer = Layer16(110, 6, 256, 128)
    gen = torch.Generator(device="cuda").manual_seed(111)
    rows = 200
    x, y = normal(gen, (rows, 256), 1.0), torch.empty((rows, 256), dtype=BF, device="cuda")
    offsets = torch.zeros(7, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_prefill_bf16_workspace_bytes(rows, 128), dtype=torch.uint8, device="cuda")
    call = lambda: moe.moe_ffn_grouped_prefill_bf16(layer.desc, x, offsets, y, ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for off in ([0, 200, 200, 200, 200, 200, 200], [0, 0, 3, 140, 140, 199, 200], [0, 33, 66, 99, 132, 165, 200]):
        offsets.copy_(torch.tensor(off, dtype=torch.int32))
        x.copy_(normal(gen, (rows, 256), 1.0))
        g.replay()
        torch.cuda.synchronize()
        for e in range(6):
            a, b = off[e], off[e + 1]
            if b > a:
                want, tol = layer.rows(e, x[a:b])[0][:2]
                check_close(y[a:b], want, tol + 2.0 ** -8 * (want.abs() + tol), f"{off} expert {e}")


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [3, 16])
def test_decode_layer_equals_the_prefill_chain_and_the_linears(T):
    """One layer two ways, as a server runs it: the decode layer with its gated shared expert and residual, and
    router -> permute -> grouped FFN -> combine with the shared expert as two linears that end on the residual."""
    E, k, H, F = 64, 6, 512, 256
    layer = Layer16(120, E + 1, H, F)
    gen = torch.Generator(device="cuda").manual_seed(121)
    wr, r, x = normal(gen, (E, H), H ** -0.5), normal(gen, (T, H), 1.0), normal(gen, (T, H), 1.0)
    y, idx, w, lg = run_decode(layer, x, k, 1, wr=wr, residual=r)

    idx2 = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w2 = torch.empty((T, k), device="cuda")
    rws = torch.zeros(moe.moe_router_route_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    moe.moe_router_route(x, wr, k, idx2, w2, rws)
    assert torch.equal(idx, idx2)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    counts, offsets, srows, inv = i32(E), i32(E + 1), i32(T * k), i32(T * k)
    xp, yp = torch.empty((T * k, H), dtype=BF, device="cuda"), torch.empty((T * k, H), dtype=BF, device="cuda")
    pws = torch.empty(moe.moe_permute_workspace_bytes(T, k, E), dtype=torch.uint8, device="cuda")
    moe.moe_permute(idx2, E, counts, offsets, srows, inv, pws, x=x, x_perm=xp)
    fws = torch.empty(moe.moe_prefill_bf16_workspace_bytes(T * k, F), dtype=torch.uint8, device="cuda")
    routed = moe.make_bf16_layer(E, H, F, layer.gu, layer.dn)
    moe.moe_ffn_grouped_prefill_bf16(routed, xp, offsets, yp, fws)
    out = torch.empty((T, H), dtype=BF, device="cuda")
    moe.moe_unpermute_combine(yp, w2, out, inv=inv)
    h = torch.empty((T, F), dtype=BF, device="cuda")
    moe.moe_linear(x, layer.gu[E], h, act=moe.MOE_ACT_SILU, gated=True)
    moe.moe_linear(h, layer.dn[E], out, residual=out)
    total = torch.empty((T, H), dtype=BF, device="cuda")
    total.copy_((out.float() + r.float()).to(BF))
    torch.cuda.synchronize()
    assert moe.moe_device_error() == 0
    ffn_close(total.float().cpu().numpy(), y.float().cpu().numpy(), "prefill chain against the decode layer")
    want, tol, _, _ = reference(layer, x, lg, k, 1, None, r)
    check_close(y, want, tol, "decode layer")


@pytest.mark.parametrize("T", [1, 4, 7])
@pytest.mark.parametrize("up, down", [(-1, 1), (-1, -1), (1, -1)])
def test_decode_infinite_input_keeps_its_sign(T, up, down):
    """An infinite h is infinite in both halves that enter the down projection, with its sign in both: y is inf of
    the product's sign, never NaN.  The down rows sum to 3 and more, so a half of the other sign would show."""
    H, F = 192, 128
    layer = Layer16(197, 8, H, F)
    layer.gu.abs_().add_(0.01)
    layer.dn.abs_().add_(0.01)
    layer.gu[:, F:] *= up
    layer.dn.mul_(down)
    layer.dn[:, 0] *= 300  # one output whose weights are large
    gen = torch.Generator(device="cuda").manual_seed(198)
    lg = torch.randn((T, 8), generator=gen, device="cuda")
    for at in (0, 100, H - 1):
        x = normal(gen, (T, H), 1.0).abs_()
        x[T - 1, at] = float("inf")
        y, _, _, _ = run_decode(layer, x, 2, lg=lg)
        assert torch.isinf(y[T - 1]).all() and (y[T - 1] * (up * down) > 0).all(), at
        assert torch.isfinite(y[: T - 1]).all(), at


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("h, w", [(-2.0 ** 128, 4.0), (2.0 ** 128, -4.0), (-2.0 ** 128, -2.0 ** 127), (2.0 ** 128, 2.0 ** -100)])
def test_decode_one_infinite_feature(T, h, w):
    """silu(2^64) = 2^64 times an up of +-2^64 is past fp32: h = +-inf in one feature, and y = inf of the sign of h w."""
    H, F = 128, 64
    layer = Layer16(199, 4, H, F)
    layer.gu.zero_()
    layer.dn.zero_()
    layer.gu[:, 0, 0] = 1.0
    layer.gu[:, F, 1] = math.copysign(2.0 ** 64, h)
    layer.dn[:, :, 0] = w
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[:, 0] = 2.0 ** 64
    x[:, 1] = 1.0
    y, _, _, _ = run_decode(layer, x, 1, lg=torch.zeros((T, 4), device="cuda"))
    assert torch.equal(y, torch.full_like(y, math.copysign(math.inf, h * w)))


def test_bindings_refuse_one_spoilt_tensor_of_a_valid_call():
    """The valid call runs; with one tensor of another type of the same bytes, of another size, with gaps or on the CPU it
    is refused, and nothing is written."""
    layer = Layer16(210, 9, 128, 64)
    gen = torch.Generator(device="cuda").manual_seed(211)
    T, k = 2, 2
    full = lambda shape, v, dt: torch.full(shape, v, dtype=dt, device="cuda")
    dec = dict(x=normal(gen, (T, 128), 1.0), y=full((T, 128), 7.0, BF), wr=normal(gen, (8, 128), 0.1), logits=full((T, 8), 7.0, torch.float32),
               shared_gate=normal(gen, (128,), 0.1), residual=normal(gen, (T, 128), 1.0),
               idx=full((T, k), -7, torch.int32), w=full((T, k), 7.0, torch.float32))
    ws = workspace(layer, T, k, 1)
    grp = dict(x_perm=normal(gen, (4, 128), 1.0), offsets=torch.tensor([0, 1, 1, 1, 4, 4, 4, 4, 4, 4], dtype=torch.int32, device="cuda"),
               y_perm=full((4, 128), 7.0, BF))
    gws = torch.zeros(moe.moe_prefill_bf16_workspace_bytes(4, 64), dtype=torch.uint8, device="cuda")
    calls = [(dec, ("y", "logits", "idx", "w"), lambda desc=layer.desc, **a: moe.moe_decode_layer_bf16(desc, k=k, ws=ws, shared=1, **a)),
             (grp, ("y_perm",), lambda desc=layer.desc, **a: moe.moe_ffn_grouped_prefill_bf16(desc, ws=gws, **a))]
    away = moe.make_bf16_layer(9, 128, 64, layer.gu, layer.dn)
    away.device += 1
    for args, outs, call in calls:
        for name, t in args.items():
            other = {BF: torch.float16, torch.float32: torch.int32, torch.int32: torch.float32}[t.dtype]
            for bad in (t.view(other), t[..., 1:].contiguous(), torch.cat([t, t]), torch.stack([t, t], -1)[..., 0], t.cpu()):
                with pytest.raises(moe.MoeError) as ei:
                    call(**{**args, name: bad})
                assert ei.value.status == moe.MOE_ERR_INVALID_ARG, name
        with pytest.raises(moe.MoeError):
            call(desc=away, **args)
        torch.cuda.synchronize()
        for o in outs:
            assert (args[o].abs() == 7).all(), o
        call(**args)
        torch.cuda.synchronize()
        for o in outs:
            assert not (args[o].abs() == 7).all(), o
    assert moe.moe_device_error() == 0


@pytest.mark.parametrize("E, H, F", [(9, 128, 128), (9, 192, 64), (10, 128, 64)])
def test_make_bf16_layer_refuses_weights_of_another_shape(E, H, F):
    layer = Layer16(212, 9, 128, 64)
    moe.make_bf16_layer(8, 128, 64, layer.gu, layer.dn)
    with pytest.raises(moe.MoeError):
        moe.make_bf16_layer(E, H, F, layer.gu, layer.dn)
    for gu, dn in [(layer.gu.cpu(), layer.dn), (layer.gu, layer.dn.cpu()), (layer.gu.half(), layer.dn), (layer.gu, layer.dn.float())]:
        with pytest.raises(moe.MoeError):
            moe.make_bf16_layer(9, 128, 64, gu, dn)


def test_bits_of_bf16_in_integer_tensors():
    """int16 and uint16 tensors of bf16 bits, for any argument, give the same call."""
    layer = Layer16(213, 4, 128, 64)
    gen = torch.Generator(device="cuda").manual_seed(214)
    x, lg = normal(gen, (3, 128), 1.0), torch.randn((3, 4), generator=gen, device="cuda")
    want = run_decode(layer, x, 2, lg=lg)[0]
    desc = moe.make_bf16_layer(4, 128, 64, layer.gu.view(torch.uint16), layer.dn.view(torch.int16))
    y = torch.empty_like(want)
    moe.moe_decode_layer_bf16(desc, x.view(torch.uint16), 2, y.view(torch.int16), workspace(layer, 3, 2, 0), logits=lg)
    assert torch.equal(y, want)


# the limits that the header names: 16 tokens up to H = 5120, one token's x up to 166,000 bytes, F = 2^20, 256 rows
@pytest.mark.parametrize("T,E,k,H,F,shared", [
    (16, 8, 4, 5120, 128, "gated"), (16, 16, 15, 5120, 64, "one"), (1, 2, 1, 82944, 64, "none"),
    (1, 1, 1, 64, 1 << 20, "none"), (2, 2, 2, 64, 1 << 18, "one"), (16, 256, 15, 64, 64, "one")])
def test_decode_layer_at_its_limits(T, E, k, H, F, shared):
    check_decode(5, T, E, k, H, F, shared, True, True)


@pytest.mark.parametrize("T", [3, 16])
def test_decode_nan_token_leaves_the_others(T):
    """A token of NaN (the padding of a batch) makes its own output NaN and no other's anything else."""
    layer = Layer16(220, 33, 256, 128)
    gen = torch.Generator(device="cuda").manual_seed(221)
    x, wr, gate = normal(gen, (T, 256), 1.0), normal(gen, (32, 256), 0.06), normal(gen, (256,), 0.06)
    y0 = run_decode(layer, x, 4, 1, wr=wr, gate=gate)[0]
    x[1] = float("nan")
    y1 = run_decode(layer, x, 4, 1, wr=wr, gate=gate)[0]
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(y0[keep], y1[keep]) and torch.isnan(y1[1]).all()
    assert moe.moe_device_error() == 0


def test_a_server_s_step_on_three_streams_at_once():
    """Decode layer, linears and grouped FFN in one graph per stream, each with its own workspaces, replayed at once:
    the same bits as one after another."""
    E, k, H, F = 64, 6, 512, 256
    layer = Layer16(230, E + 1, H, F)

    def state(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        empty = lambda *shape: torch.empty(shape, dtype=BF, device="cuda")
        offsets = torch.tensor([700 * i // (E + 1) for i in range(E + 2)], dtype=torch.int32, device="cuda")
        return dict(x=normal(gen, (7, H), 1.0), wr=normal(gen, (E, H), H ** -0.5), ws=workspace(layer, 7, k, 1), y=empty(7, H),
                    gx=normal(gen, (700, H), 1.0), off=offsets, gy=empty(700, H), lw=normal(gen, (2048, H), 0.05),
                    gws=empty(700, F), ly=empty(700, 2048), ly2=empty(7, 2048))

    def step(s):
        moe.moe_decode_layer_bf16(layer.desc, s["x"], k, s["y"], s["ws"], wr=s["wr"], shared=1)
        moe.moe_linear(s["y"], s["lw"], s["ly2"])
        moe.moe_ffn_grouped_prefill_bf16(layer.desc, s["gx"], s["off"], s["gy"], s["gws"])
        moe.moe_linear(s["gy"], s["lw"], s["ly"], act=moe.MOE_ACT_GELU)
        moe.moe_decode_layer_bf16(layer.desc, s["y"], k, s["x"], s["ws"], wr=s["wr"], shared=1)

    alone, at_once = [state(i) for i in range(3)], [state(i) for i in range(3)]
    for s in alone:
        for _ in range(6):
            step(s)
            torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in range(3)], []
    for s, q in zip(at_once, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=q):
            for _ in range(3):
                step(s)
    torch.cuda.synchronize()
    for _ in range(2):
        for g, q in zip(graphs, streams):
            with torch.cuda.stream(q):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(alone, at_once):
        assert all(torch.equal(a[n], b[n]) for n in ("x", "y", "gy", "ly", "ly2"))
    assert moe.moe_device_error() == 0
