"""GPU parity of moe_linear against the definition in 64 bits.

Small integers make every product and partial sum an exact fp32 value whatever
the order, so those tests ask for equality.  On random values the tolerance
counts, per element:
  - the fp32 sum: K products in any order, each addition off by at most one
    unit in the last place: A = (K + 2) 2^-23 (sum |x||w| + |bias|);
  - the activation: its slope (at most 1.2 for all of them) times A, and its own
    evaluation, at most 2^-19 of the larger of its value and 2^-2 (the
    error of exp at |argument| <= 32: 2 + 1.2 * 32 ulps of 2^-23);
  - for gated products both factors' errors times the other factor;
  - one fp32 rounding of each of the remaining steps (2^-22 of the values), and
    the final rounding: eps / 2 of the value (plus half the smallest f16
    subnormal, 2^-25).
"""
import pytest
import torch

import quantized_moe_route_b200 as moe

pytestmark = pytest.mark.gpu

ACTS = {"none": lambda v: v, "silu": lambda v: v * torch.special.expit(v),
        "gelu": lambda v: v * torch.special.ndtr(v),
        "gelu_tanh": lambda v: 0.5 * v * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3))),
        "relu": lambda v: v.clamp(min=0), "sigmoid": torch.special.expit}
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def act_id(name):
    return getattr(moe, "MOE_ACT_" + name.upper())


def padded(rows, cols, ld, dtype, fill=float("nan")):
    """A [rows][cols] view of a wider buffer whose tails hold `fill`."""
    buf = torch.full((rows, ld), fill, dtype=dtype, device="cuda")
    return buf, buf[:, :cols]


def ints(gen, shape, dtype, lim=3):
    return torch.randint(-lim, lim + 1, shape, generator=gen, device="cuda").to(dtype)


def up8(k):
    return (k + 7) // 8 * 8


# T around the tile and token-group edges, N and K odd, tiny, and past the tiles
EXACT = [(1, 1, 1), (1, 16, 8), (1, 2048, 2048), (2, 5, 7), (3, 100, 40), (4, 17, 72), (7, 512, 2048), (8, 129, 100),
         (9, 1000, 512), (13, 4099, 1000), (15, 300, 264), (16, 2048, 2048), (16, 33, 4104), (5, 24, 16384),
         (1, 7, 40000), (17, 128, 64), (17, 127, 2050), (31, 257, 33), (33, 2049, 96), (64, 512, 2048), (100, 96, 8200),
         (127, 640, 129), (128, 128, 128), (129, 2048, 512), (200, 130, 65), (255, 1, 1000), (256, 256, 256),
         (257, 385, 640), (300, 5, 15), (513, 1025, 320), (1000, 264, 192), (2050, 384, 72)]


@pytest.mark.parametrize("T,N,K", EXACT)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_integers_are_exact(T, N, K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T * 131 + N * 17 + K)
    dt = DT[dtype]
    _, x = padded(T, K, up8(K) + 8 * (T % 3), dt)
    _, w = padded(N, K, up8(K) + 8 * (N % 2), dt)
    x.copy_(ints(gen, (T, K), dt))
    w.copy_(ints(gen, (N, K), dt))
    bias = ints(gen, (N,), dt, 50)
    ybuf, y = padded(T, N, N + 5, torch.float32, 777.0)
    moe.moe_linear(x, w, y, bias=bias)
    want = x.double() @ w.double().t() + bias.double()
    assert torch.equal(y.double(), want)
    assert (ybuf[:, N:] == 777.0).all(), "wrote past the row"
    # 16-bit output: the exact value rounded once, on a residual that y replaces
    rbuf, r = padded(T, N, N + 3, dt, 5.0)
    r.copy_(ints(gen, (T, N), dt, 100))
    want16 = (want + r.double()).float().to(dt)
    moe.moe_linear(x, w, r, bias=bias, residual=r)
    assert torch.equal(r, want16)
    assert (rbuf[:, N:] == 5.0).all()


@pytest.mark.parametrize("T,N,K", [(1, 512, 2048), (3, 13, 24), (9, 65, 136), (16, 1000, 520), (40, 64, 72), (130, 200, 300),
                                   (300, 512, 2048), (700, 129, 65)])
def test_gated_integers_are_exact(T, N, K):
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    dt = torch.float16
    _, x = padded(T, K, up8(K), dt)
    x.copy_(ints(gen, (T, K), dt, 2))
    w = torch.zeros((2 * N, up8(K)), dtype=dt, device="cuda")[:, :K]
    w.copy_(ints(gen, (2 * N, K), dt, 2))
    bias = ints(gen, (2 * N,), dt)
    y = torch.empty((T, N), dtype=torch.float32, device="cuda")
    moe.moe_linear(x, w, y, bias=bias, act=moe.MOE_ACT_RELU, gated=True)
    v = x.double() @ w.double().t() + bias.double()
    want = v[:, :N].clamp(min=0) * v[:, N:]
    assert want.abs().max() < 2 ** 24
    assert torch.equal(y.double(), want)


def check_random(T, N, K, dtype, act, gated, bias, residual, out32, pad, seed, ldy=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, rows = DT[dtype], 2 * N if gated else N
    _, x = padded(T, K, up8(K) + pad, dt)
    _, w = padded(rows, K, up8(K) + pad, dt)
    x.copy_(torch.randn((T, K), generator=gen, device="cuda"))
    w.copy_(torch.randn((rows, K), generator=gen, device="cuda") * K ** -0.5)
    b = (0.5 * torch.randn(rows, generator=gen, device="cuda")).to(dt) if bias else None
    r = torch.randn((T, ldy or N + pad), generator=gen, device="cuda").to(dt)[:, :N] if residual else None
    ybuf, y = padded(T, N, ldy or N + pad + 1, torch.float32 if out32 else dt, 3.0)
    moe.moe_linear(x, w, y, bias=b, residual=r, act=act_id(act), gated=gated)
    xd, wd = x.double(), w.double()
    bd = b.double() if bias else torch.zeros(rows, dtype=torch.float64, device="cuda")
    v = xd @ wd.t() + bd
    A = (K + 2) * 2.0 ** -23 * (xd.abs() @ wd.abs().t() + bd.abs())
    a = ACTS[act](v[:, :N])
    Ea = 1.2 * A[:, :N] + (0 if act in ("none", "relu") else 2.0 ** -19 * a.abs().clamp(min=0.25))
    if gated:
        u = v[:, N:]
        want = a * u
        tol = Ea * (u.abs() + A[:, N:]) + a.abs() * A[:, N:] + 2.0 ** -22 * want.abs()
    else:
        want, tol = a, Ea
    if residual:
        want = want + r.double()
        tol = tol + 2.0 ** -22 * (want.abs() + r.double().abs())
    if not out32:
        tol = tol + torch.finfo(dt).eps / 2 * (want.abs() + tol) + 2.0 ** -25
    err = (y.double() - want).abs()
    assert (err <= tol).all(), f"worst {((err - tol).max()):.3e} past the bound"
    # the same on the whole: rounding to the output type, and the fp32 sums
    # (2^-20 of the values, far above sqrt(K) 2^-24)
    rel = (err.norm() / want.norm()).item()
    assert rel <= (2.0 ** -20 if out32 else torch.finfo(dt).eps / 2), rel
    assert (ybuf[:, N:] == 3.0).all()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,N,K,dtype,out32", [(1, 512, 2048, "bf16", False), (6, 77, 136, "f16", True),
                                               (16, 300, 1000, "bf16", True), (90, 200, 264, "f16", False),
                                               (300, 513, 2048, "bf16", False)])
def test_random_values(T, N, K, dtype, out32, act, gated):
    check_random(T, N, K, dtype, act, gated, True, True, out32, 8, T + N)


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("T", [1, 12, 60, 400])
def test_optional_terms(T, bias, residual):
    check_random(T, 384, 512, "bf16", "silu", False, bias, residual, False, 0, T)
    check_random(T, 200, 512, "f16", "gelu", True, bias, residual, True, 16, T + 1)


def test_same_bits_every_call_and_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(1)
    for T, N, K in [(3, 512, 2048), (48, 256, 4096), (400, 1000, 512)]:
        x = torch.randn((T, K), generator=gen, device="cuda").bfloat16()
        w = torch.randn((N, K), generator=gen, device="cuda").bfloat16()
        ys = [torch.empty((T, N), device="cuda") for _ in range(4)]
        moe.moe_linear(x, w, ys[0])
        moe.moe_linear(x, w, ys[1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        moe.moe_linear(x, w, ys[2], stream=s)
        with torch.cuda.stream(s):
            moe.moe_linear(x, w, ys[3])
        torch.cuda.synchronize()
        assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_two_calls_at_once_on_two_streams():
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = [ints(gen, (40, 2048), torch.bfloat16) for _ in range(2)]
    w = [ints(gen, (2048, 2048), torch.bfloat16) for _ in range(2)]
    y = [torch.empty((40, 2048), device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            moe.moe_linear(x[i], w[i], y[i], stream=streams[i])
            moe.moe_linear(x[i][:3], w[i], y[i][:3], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(y[i].double(), x[i].double() @ w[i].double().t())


def test_captured_chain_replays_on_new_inputs():
    """A shared expert as two linears in one graph: gated up, then down onto the residual stream in place."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, H, F = 5, 512, 256
    x, wu, wd = ints(gen, (T, H), torch.bfloat16, 1), ints(gen, (2 * F, H), torch.bfloat16, 1), ints(
        gen, (H, F), torch.bfloat16, 1)
    h, r = torch.empty((T, F), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda").bfloat16()
    y = torch.empty((T, H), device="cuda")

    def chain():
        moe.moe_linear(x, wu, h, act=moe.MOE_ACT_RELU, gated=True)
        moe.moe_linear(h, wd, y, residual=r)

    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for seed in range(3):
        x.copy_(ints(gen, (T, H), torch.bfloat16, 1))
        r.copy_(ints(gen, (T, H), torch.bfloat16, 9))
        g.replay()
        torch.cuda.synchronize()
        v = x.double() @ wu.double().t()
        hh = (v[:, :F].clamp(min=0) * v[:, F:]).float().bfloat16()
        # |h| < 2^8 * 2^7 holds 8 bits each; sums of F values of at most 2^15 in steps of 2^0 stay exact below 2^24
        assert torch.equal(h, hh)
        assert torch.equal(y.double(), hh.double() @ wd.double().t() + r.double())


@pytest.mark.parametrize("T", [2, 20])
def test_offsets_past_32_bits(T):
    """Rows of w, x, y and residual so far apart that element offsets pass 2^31."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    N, K, far = 40, 72, (1 << 31) // 32 + 8
    w = torch.empty(far * (N - 1) + K, dtype=torch.bfloat16, device="cuda").as_strided((N, K), (far, 1))
    xs = (1 << 31) // (T - 1) + 8
    xs += -xs % 8
    x = torch.empty(xs * (T - 1) + K, dtype=torch.bfloat16, device="cuda").as_strided((T, K), (xs, 1))
    y = torch.empty(xs * (T - 1) + N, dtype=torch.bfloat16, device="cuda").as_strided((T, N), (xs, 1))
    w.copy_(ints(gen, (N, K), torch.bfloat16))
    x.copy_(ints(gen, (T, K), torch.bfloat16))
    y.copy_(ints(gen, (T, N), torch.bfloat16))
    want = (x.double() @ w.double().t() + y.double()).float().bfloat16()
    moe.moe_linear(x, w, y, residual=y)
    assert torch.equal(y, want)


def test_infinite_and_large_values_keep_their_meaning():
    """Values past the f16 range round to infinity; silu and sigmoid reach their limits at +-large."""
    K = 64
    x = torch.ones((3, K), dtype=torch.float16, device="cuda")
    x[1] = -1
    x[2] = 0
    w = torch.full((20, K), 1200.0, dtype=torch.float16, device="cuda")
    y = torch.empty((3, 20), dtype=torch.float16, device="cuda")
    moe.moe_linear(x, w, y)
    assert torch.isposinf(y[0]).all() and torch.isneginf(y[1]).all() and (y[2] == 0).all()
    for act, lims in (("silu", (float("inf"), 0.0, 0.0)), ("sigmoid", (1.0, 0.0, 0.5)), ("gelu", (float("inf"), 0.0, 0.0)),
                      ("gelu_tanh", (float("inf"), 0.0, 0.0)), ("relu", (float("inf"), 0.0, 0.0))):
        moe.moe_linear(x, w, y, act=act_id(act))
        for t in range(3):
            assert (y[t] == lims[t]).all(), act


def test_empty_calls_write_nothing():
    x, w = torch.ones((4, 16), device="cuda").bfloat16(), torch.ones((8, 16), device="cuda").bfloat16()
    y = torch.full((4, 8), 9.0, device="cuda")
    moe.moe_linear(x[:0], w, y[:0])
    moe.moe_linear(x, w[:0], y[:, :0])
    torch.cuda.synchronize()
    assert (y == 9.0).all()


def test_non_finite_rows_stay_in_their_rows():
    """Infinities and NaN in a row of x, or of w, reach that row's (that output's) results and no others."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    for T, N, K in [(5, 40, 136), (13, 300, 520), (100, 300, 520), (700, 1024, 200)]:
        x, w = ints(gen, (T, K), torch.bfloat16), ints(gen, (N, K), torch.bfloat16)
        y0, y1 = torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
        moe.moe_linear(x, w, y0)
        x[T // 2, 3], x[1, K - 1], w[N - 1, 0] = float("nan"), float("inf"), float("-inf")
        moe.moe_linear(x, w, y1)
        keep = torch.ones((T, N), dtype=torch.bool, device="cuda")
        keep[T // 2], keep[1], keep[:, N - 1] = False, False, False
        assert torch.equal(y0[keep], y1[keep])
        assert torch.isnan(y1[T // 2]).all() and not torch.isfinite(y1[1][w[:, K - 1] != 0]).any()


@pytest.mark.parametrize("which", ["linear", "decode", "grouped"])
def test_first_call_of_a_process_inside_a_capture(which):
    """Attributes, maps and occupancy are looked up on the first call, which may be a captured one."""
    import os
    import subprocess
    import sys
    code = f"""
import sys
sys.path.insert(0, {os.path.dirname(os.path.dirname(os.path.abspath(__file__)))!r})
import torch
import quantized_moe_route_b200 as moe
bf = torch.bfloat16
gu, dn = torch.ones((4, 128, 64), dtype=bf, device="cuda") / 64, torch.ones((4, 64, 64), dtype=bf, device="cuda") / 64
layer = moe.make_bf16_layer(4, 64, 64, gu, dn)
x, y = torch.ones((40, 64), dtype=bf, device="cuda"), torch.zeros((40, 64), dtype=bf, device="cuda")
off = torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32, device="cuda")
ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
lg = torch.zeros((4, 4), device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    if {which!r} == "linear":
        moe.moe_linear(x, gu[0, :64], y)
        moe.moe_linear(x[:4], gu[0, :64], y[:4])
    elif {which!r} == "decode":
        moe.moe_decode_layer_bf16(layer, x[:4], 2, y[:4], ws, logits=lg)
    else:
        moe.moe_ffn_grouped_prefill_bf16(layer, x, off, y, ws)
g.replay()
torch.cuda.synchronize()
s = 1 / (1 + torch.tensor(-1.0).exp())  # g = u = 1, h = silu(1), y = h
want = 1.0 if {which!r} == "linear" else s.item()
assert (y[:4].float() - want).abs().max() < 0.01, y
assert moe.moe_device_error() == 0
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


@pytest.mark.parametrize("T,N,K,gated", [(20, 130, 4096, False), (333, 1500, 2048, False), (1000, 2050, 4096, False),
                                         (300, 700, 4096, True), (40, 128, 16384, False)])
def test_long_sums_keep_fp32_accuracy(T, N, K, gated):
    """fp32 outputs of long sums: 2^-20 of the values as a whole (check_random's bound), whatever K."""
    check_random(T, N, K, "bf16", "none", gated, True, False, True, 0, T + K)


# tiles for all SMs: rows on M (alone, K < 1024; on pairs of SMs, K >= 1024), ragged in rows, outputs and K
@pytest.mark.parametrize("T,N,K,dtype,gated,pad", [
    (2432, 2048, 64, "bf16", False, 0), (1921, 2049, 136, "f16", False, 0), (9000, 300, 520, "f16", True, 3),
    (20000, 250, 72, "bf16", False, 0), (2500, 2048, 1024, "bf16", False, 0), (2433, 2047, 1096, "f16", False, 5),
    (2700, 1300, 1032, "bf16", True, 0), (129 * 128, 130, 1025, "bf16", False, 1), (4225, 1200, 2048, "f16", False, 8)])
def test_large_products_are_exact_on_integers(T, N, K, dtype, gated, pad):
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    dt, rows = DT[dtype], 2 * N if gated else N
    _, x = padded(T, K, up8(K) + 8 * (T % 2), dt)
    _, w = padded(rows, K, up8(K), dt)
    x.copy_(ints(gen, (T, K), dt, 1))
    w.copy_(ints(gen, (rows, K), dt, 1))
    bias = ints(gen, (rows,), dt, 2)
    rbuf, r = padded(T, N, N + pad, dt, 5.0)
    r.copy_(ints(gen, (T, N), dt, 9))
    v = x.double() @ w.double().t() + bias.double()
    want = (v[:, :N].clamp(min=0) * v[:, N:] if gated else v.clamp(min=0)) + r.double()
    moe.moe_linear(x, w, r, bias=bias, residual=r, act=moe.MOE_ACT_RELU, gated=gated)  # in place
    assert torch.equal(r, want.float().to(dt))
    assert (rbuf[:, N:] == 5.0).all()
    assert moe.moe_device_error() == 0


@pytest.mark.parametrize("act,gated", [("gelu_tanh", False), ("silu", True), ("gelu", True)])
def test_large_products_random(act, gated):
    check_random(2600, 1100, 1200, "bf16", act, gated, True, True, False, 8, 5)
    check_random(4200, 1111, 200, "f16", act, gated, True, True, False, 8, 6)


# large products whose rows of y are no whole vectors (weights on M), and fp32 outputs in tiles of up to 192 rows
@pytest.mark.parametrize("T,N,K,out32,gated", [
    (2600, 1101, 1200, False, False), (1500, 5002, 520, False, False), (2600, 555, 520, False, True),
    (333, 8192, 1032, True, False), (2048, 5000, 520, True, False), (333, 2048, 4096, True, True), (2000, 1001, 520, True, True)])
def test_large_products_in_other_tiles(T, N, K, out32, gated):
    check_random(T, N, K, "bf16", "silu", gated, True, True, out32, 0, T + N)


# rows on M (alone, K < 1024; on pairs of SMs, K >= 1024): rows of y and of the residual on 16 bytes, N whatever
@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
@pytest.mark.parametrize("T,N,K,dtype,gated", [
    (2600, 1101, 1200, "bf16", False), (4200, 1111, 200, "f16", False), (2048, 2048, 512, "bf16", False),
    (2600, 1001, 1100, "bf16", True), (1500, 907, 264, "f16", True)])
def test_large_products_rows_on_m(T, N, K, dtype, gated, act):
    check_random(T, N, K, dtype, act, gated, True, True, False, 8, T + N, ldy=N + 15 - (N + 7) % 8)


def test_large_product_with_unaligned_residual():
    gen = torch.Generator(device="cuda").manual_seed(13)
    T, N, K = 2048, 2048, 256
    x, w = ints(gen, (T, K), torch.bfloat16, 1), ints(gen, (N, K), torch.bfloat16, 1)
    r = ints(gen, (T, N + 2), torch.bfloat16)[:, 1:N + 1]
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_linear(x, w, y, residual=r)
    want = x.double() @ w.double().t() + r.double()
    assert want.abs().max() <= 256  # exact in bf16
    assert torch.equal(y.double(), want)


def test_large_products_same_bits_and_captured():
    gen = torch.Generator(device="cuda").manual_seed(12)
    x, w = torch.randn((2560, 1024), generator=gen, device="cuda").bfloat16(), torch.randn((2048, 1024), generator=gen, device="cuda").bfloat16()
    ys = [torch.empty((2560, 2048), device="cuda").bfloat16() for _ in range(3)]
    moe.moe_linear(x, w, ys[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):  # two at once
        for s, y in zip(streams, ys[1:]):
            moe.moe_linear(x, w, y, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_linear(x, w, ys[1])
        moe.moe_linear(x, w, ys[2], residual=ys[1])
    x.copy_(torch.randn((2560, 1024), generator=gen, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    moe.moe_linear(x, w, ys[0])
    assert torch.equal(ys[0], ys[1])
    moe.moe_linear(x, w, ys[0], residual=ys[0])
    assert torch.equal(ys[0], ys[2]) and moe.moe_device_error() == 0


# the weight stream (up to 16 and 32 rows), tiles alone and with K over a cluster, rows on M alone and on pairs of SMs
NAN_SIZES = [(5, 40, 136), (24, 300, 1024), (100, 300, 200), (100, 300, 2048), (2500, 2048, 136), (2500, 2048, 1024)]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("T,N,K", NAN_SIZES)
def test_nan_passes_every_activation(T, N, K, out32, gated, act):
    """A NaN in a row of x, in a row of w (gated: of the gate or of the up half) or in the bias makes that row or that
    output NaN under every activation, and leaves all others their bits."""
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    bf, rows = torch.bfloat16, 2 * N if gated else N
    x = torch.randn((T, K), generator=gen, device="cuda").to(bf)
    w = (torch.randn((rows, K), generator=gen, device="cuda") * K ** -0.5).to(bf)
    b = torch.randn(rows, generator=gen, device="cuda").to(bf)
    ys = [torch.empty((T, N), dtype=torch.float32 if out32 else bf, device="cuda") for _ in range(2)]
    call = lambda y: moe.moe_linear(x, w, y, bias=b, act=act_id(act), gated=gated)
    call(ys[0])
    nan = float("nan")
    x[T // 2, 3], w[1, K - 1], w[rows - 2, 0], b[7], b[rows - 9] = nan, nan, nan, nan, nan
    call(ys[1])
    hit = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    hit[T // 2] = True
    hit[:, [1, N - 2, 7, N - 9]] = True
    assert torch.isnan(ys[1][hit]).all()
    assert torch.equal(ys[0][~hit], ys[1][~hit])


@pytest.mark.parametrize("act,lo", [("silu", -60.0), ("sigmoid", -60.0), ("gelu", -9.0), ("gelu_tanh", -9.0)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,N,K", [(16, 33, 1), (200, 40, 1), (100, 300, 2048), (2500, 2048, 64), (2500, 2048, 1024)])
def test_activations_keep_their_relative_accuracy_in_the_tail(T, N, K, out, gated, act, lo):
    """Arguments v below zero that arrive exactly (one input of x is v, its weight 1, all else 0; gated: up is 1).
    In units of 2^-23 of the value: 16 for the functions and operations themselves (GELU's fit: 2^-20.3), the rounded
    argument z of exp (v^2 / 2 within one half each of two roundings; 2 z' of tanh within 4), and for 16-bit results
    __expf's documented 2 + 1.2 |z| and 4 for its division; then the result's rounding."""
    dt = torch.float16 if out == "f16" else torch.bfloat16
    rows = 2 * N if gated else N
    v = torch.linspace(lo, -0.25, T, device="cuda").to(dt)
    x = torch.zeros((T, up8(K)), dtype=dt, device="cuda")[:, :K]
    x[:, K // 2] = v
    w = torch.zeros((rows, up8(K)), dtype=dt, device="cuda")[:, :K]
    w[:N, K // 2] = 1
    b = torch.zeros(rows, dtype=dt, device="cuda")
    b[N:] = 1
    y = torch.empty((T, N), dtype=torch.float32 if out == "f32" else dt, device="cuda")
    moe.moe_linear(x, w, y, bias=b, act=act_id(act), gated=gated)
    v = v.double()
    if act == "gelu_tanh":  # 1 + tanh cancels in 64 bits too: 1 / (1 + exp(-2 z))
        z = 2 * (2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3)
        want, ulps = v * torch.special.expit(z), 16 + 4 * z.abs()
    else:
        z = -v * v / 2 if act == "gelu" else v
        # (erfc, since ndtr is 0 in the tail)
        want = v * 0.5 * torch.special.erfc(-v * 0.5 ** 0.5) if act == "gelu" else ACTS[act](v)
        ulps = 16 + (z.abs() if act == "gelu" else 0)
    if out != "f32":
        ulps = ulps + 6 + 1.2 * z.abs()
    tol = ulps * 2.0 ** -23 * want.abs()
    if out != "f32":
        tol = tol + torch.finfo(dt).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if out == "f16" else 0)
    err = (y.double() - want.unsqueeze(1)).abs()
    assert (err <= tol.unsqueeze(1)).all(), f"worst {(err.max(1).values / tol).max().item():.2f} of the bound"


def test_bits_of_bf16_in_integer_tensors():
    """bf16 tensors and int16 or uint16 tensors of bf16 bits, mixed, give the same call."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    bf = torch.bfloat16
    x, w, b, r = ints(gen, (20, 72), bf), ints(gen, (24, 72), bf), ints(gen, (24,), bf), ints(gen, (20, 24), bf)
    want, y = torch.empty((20, 24), dtype=bf, device="cuda"), torch.empty((20, 24), dtype=bf, device="cuda")
    moe.moe_linear(x, w, want, bias=b, residual=r)
    i16, u16 = torch.int16, torch.uint16
    for dx, dw, db, dr, dy in [(i16,) * 5, (u16,) * 5, (u16, bf, i16, bf, u16), (bf, u16, u16, i16, bf)]:
        y.zero_()
        moe.moe_linear(x.view(dx), w.view(dw), y.view(dy), bias=b.view(db), residual=r.view(dr))
        assert torch.equal(y, want), (dx, dw, db, dr, dy)
    y32 = torch.empty((20, 24), device="cuda")
    moe.moe_linear(x.view(u16), w, y32)
    assert torch.equal(y32.double(), x.double() @ w.double().t())
    for bad in (dict(x=x.view(torch.float16)), dict(w=w.view(torch.float16)), dict(y=y.view(torch.float16))):
        with pytest.raises(moe.MoeError):
            moe.moe_linear(**{**dict(x=x, w=w, y=y), **bad})


def test_pairs_of_sms_back_to_back_with_other_kernels():
    """The kernel on pairs of SMs in turn with the tiles and the weight stream, launches following one another closely:
    no CTA's late arrivals reach a successor (the same bits as alone)."""
    gen = torch.Generator(device="cuda").manual_seed(16)
    w = torch.randn((2048, 1024), generator=gen, device="cuda").bfloat16()
    xs = [torch.randn((T, 1024), generator=gen, device="cuda").bfloat16() for T in (2500, 2500, 300, 40, 9)]
    ys = [torch.empty((x.shape[0], 2048), dtype=torch.bfloat16, device="cuda") for x in xs]
    for x, y in zip(xs, ys):
        moe.moe_linear(x, w, y)
        torch.cuda.synchronize()
    alone = [y.clone() for y in ys]
    for y in ys:
        y.zero_()
    for _ in range(200):
        for x, y in zip(xs, ys):
            moe.moe_linear(x, w, y)
    torch.cuda.synchronize()
    assert all(torch.equal(a, y) for a, y in zip(alone, ys)) and moe.moe_device_error() == 0


@pytest.mark.parametrize("T,N,K,dtype,out32", [
    (1, 24, 16384, "bf16", True), (5, 24, 65536, "bf16", True), (16, 24, 1 << 20, "f16", True), (30, 24, 65536, "f16", True),
    (40, 24, 1 << 17, "bf16", True), (3, 24, 1 << 20, "f16", False), (40, 24, 1 << 18, "f16", False),
    (2500, 2048, 1 << 16, "f16", False), (40, 24, 1 << 20, "bf16", False)])
def test_long_sums_of_one_sign(T, N, K, dtype, out32):
    """Products of one sign, the worst case of additions that truncate: a segment of at most 512 inputs a chain takes at
    most 32 of them, 33 2^-23 with the products' own, and the additions of segments, rounded to nearest, at most 2^-24
    each.  Their directions are random, so the error as a whole stays at 2^-19; a 16-bit result has its rounding too."""
    gen = torch.Generator(device="cuda").manual_seed(T + K)
    dt = DT[dtype]
    x = torch.rand((T, K), generator=gen, device="cuda").to(dt)
    w = (torch.rand((N, K), generator=gen, device="cuda") * (4 / K if dtype == "bf16" else 1 / 256)).to(dt)
    y = torch.empty((T, N), dtype=torch.float32 if out32 else dt, device="cuda")
    moe.moe_linear(x, w, y)
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    for k in range(0, K, 1 << 14):
        want += x[:, k:k + (1 << 14)].double() @ w[:, k:k + (1 << 14)].double().t()
    rel = (y.double() - want) / want
    tol = 33 * 2.0 ** -23 + K / 512 * 2.0 ** -24
    if out32:
        assert rel.abs().max() <= tol and rel.norm() / rel.numel() ** 0.5 <= 2.0 ** -19
    else:
        assert rel.abs().max() <= torch.finfo(dt).eps / 2 + 2 * tol
