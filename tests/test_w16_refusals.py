"""Refusals and no-ops of the 16-bit-weight calls.  Argument errors are found
on the host before any launch, so all of this runs without a GPU (the
pointers are never followed)."""
import ctypes

import pytest
import torch

import quantized_moe_route_b200 as moe

INV, SHAPE, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_ERR_WORKSPACE
P, Q = 1 << 20, 1 << 30  # aligned addresses that are never followed


def linear(x=P, ldx=64, w=P, ldw=64, T=4, N=32, K=64, dtype=moe.MOE_BF16, bias=None, act=0, gated=0, residual=None,
           ldr=0, y=Q, ldy=32, y_dtype=None):
    y_dtype = dtype if y_dtype is None else y_dtype
    return moe.lib().moe_linear(x, ldx, w, ldw, T, N, K, dtype, bias, act, gated, residual, ldr, y, ldy, y_dtype, None)


@pytest.mark.parametrize("want,kw", [
    (INV, dict(T=-1)), (INV, dict(N=-1)), (INV, dict(K=0)), (INV, dict(K=-8)),
    (INV, dict(dtype=moe.MOE_F32)), (INV, dict(dtype=3)), (INV, dict(y_dtype=moe.MOE_F16)),
    (INV, dict(dtype=moe.MOE_F16, y_dtype=moe.MOE_BF16)), (INV, dict(act=-1)), (INV, dict(act=6)),
    (INV, dict(gated=2)), (INV, dict(gated=-1)),
    (INV, dict(x=None)), (INV, dict(w=None)), (INV, dict(y=None)),
    (INV, dict(ldx=56)), (INV, dict(ldw=56)), (INV, dict(ldy=31)), (INV, dict(residual=P, ldr=31)),
    (INV, dict(x=P + 8)), (INV, dict(w=P + 2)), (INV, dict(y=Q + 1)), (INV, dict(y=Q + 2, y_dtype=moe.MOE_F32)),
    (INV, dict(bias=P + 1)), (INV, dict(residual=P + 1, ldr=32)),
    (INV, dict(residual=Q, ldr=40, ldy=32)), (INV, dict(residual=Q, ldr=32, y_dtype=moe.MOE_F32)),
    (INV, dict(y=P)), (INV, dict(bias=Q)),
    (SHAPE, dict(ldx=68)), (SHAPE, dict(ldw=65)), (SHAPE, dict(ldx=(1 << 38) + 8)),
    (SHAPE, dict(T=(1 << 30) + 1)), (SHAPE, dict(K=(1 << 30) + 1, ldx=1 << 31, ldw=1 << 31)),
    (SHAPE, dict(N=(1 << 29) + 1, ldy=1 << 31)),
    (moe.MOE_OK, dict(T=0)), (moe.MOE_OK, dict(N=0)), (moe.MOE_OK, dict(T=0, x=None, w=None, y=None)),
])
def test_linear_refusals(want, kw):
    assert linear(**kw) == want


def test_linear_binding_refuses_what_the_abi_cannot_see():
    bf = torch.bfloat16
    x, w, y = torch.zeros(2, 16, dtype=bf), torch.zeros(8, 16, dtype=bf), torch.zeros(2, 8, dtype=bf)
    bad = [
        dict(y=torch.zeros(3, 8, dtype=bf)), dict(y=torch.zeros(2, 4, dtype=bf)), dict(x=x.half()),
        dict(y=y.half()), dict(bias=torch.zeros(8)), dict(bias=torch.zeros(7, dtype=bf)),
        dict(bias=torch.zeros(16, dtype=bf)[::2]), dict(residual=torch.zeros(2, 7, dtype=bf)), dict(gated=True),
        dict(x=torch.zeros(16, 2, dtype=bf).t()), dict(x=x.float(), w=w.float()),
        {},  # CPU tensors
    ]
    for kw in bad:
        a = dict(x=x, w=w, y=y)
        a.update(kw)
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_linear(**a)
        assert ei.value.status == INV, kw


def decode(E=8, H=128, F=64, gu=P, dn=P, x=P, wr=P, logits=None, T=2, k=2, shared=0, sg=None, residual=None, y=Q,
           idx=None, w=None, ws=P, ws_bytes=1 << 40):
    layer = moe.moe_bf16_layer(E, H, F, gu, dn)
    return moe.lib().moe_decode_layer_bf16(ctypes.byref(layer), x, wr, logits, T, k, shared, sg, residual, y, idx, w,
                                           ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (INV, dict(T=-1)), (INV, dict(k=0)), (INV, dict(shared=2)), (INV, dict(shared=-1)), (INV, dict(E=0)),
    (INV, dict(H=0)), (INV, dict(F=-64)), (INV, dict(k=9)), (INV, dict(k=8, shared=1)), (INV, dict(E=1, k=1, shared=1)),
    (INV, dict(sg=P)), (INV, dict(gu=None)), (INV, dict(dn=None)), (INV, dict(x=None)), (INV, dict(y=None)),
    (INV, dict(wr=None)), (INV, dict(idx=P)), (INV, dict(w=P)),
    (INV, dict(gu=P + 8)), (INV, dict(dn=P + 8)), (INV, dict(x=P + 2)), (INV, dict(wr=P + 2)), (INV, dict(y=Q + 4)), (INV, dict(y=P)),
    (INV, dict(residual=P + 2)), (INV, dict(shared=1, sg=P + 2)), (INV, dict(ws=P + 8)), (INV, dict(logits=P + 2)),
    (INV, dict(idx=P + 2, w=P)), (INV, dict(idx=P, w=P + 1)),
    (SHAPE, dict(H=96)), (SHAPE, dict(F=32)), (SHAPE, dict(T=17)), (SHAPE, dict(E=64, T=16, k=17)),
    (SHAPE, dict(E=1025)), (SHAPE, dict(E=64, T=1, k=33)), (SHAPE, dict(E=64, T=1, k=32, shared=1)),
    (SHAPE, dict(E=64, T=16, k=16, shared=1)),
    (SHAPE, dict(T=16, H=5184)), (SHAPE, dict(T=1, H=83008)), (SHAPE, dict(F=(1 << 20) + 64)),
    (WS, dict(ws=None)), (WS, dict(ws_bytes=100)), (WS, dict(T=16, H=5120, ws_bytes=100)), (moe.MOE_OK, dict(T=0)),
])
def test_decode_layer_refusals(want, kw):
    assert decode(**kw) == want


def test_decode_layer_null_struct_and_workspace_size():
    L = moe.lib()
    assert L.moe_decode_layer_bf16(None, P, P, None, 1, 1, 0, None, None, P, None, None, P, 1 << 30, None) == INV
    need = moe.moe_decode_layer_bf16_workspace_bytes(2, 2, 0, 8, 128, 64)
    assert need > 0 and decode(ws_bytes=need - 1) == WS
    for bad in [(0, 2, 0, 8, 128, 64), (2, 0, 0, 8, 128, 64), (2, 2, 2, 8, 128, 64), (2, 2, 0, 0, 128, 64),
                (2, 2, 1, 1, 128, 64), (2, 2, 0, 8, 0, 64), (2, 2, 0, 8, 128, 0)]:
        assert moe.moe_decode_layer_bf16_workspace_bytes(*bad) == 0


def grouped(E=8, H=128, F=64, gu=P, dn=P, x=P, offsets=P, rows=4, y=P, ws=P, ws_bytes=1 << 40):
    layer = moe.moe_bf16_layer(E, H, F, gu, dn)
    return moe.lib().moe_ffn_grouped_prefill_bf16(ctypes.byref(layer), x, offsets, rows, y, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (INV, dict(rows=-1)), (INV, dict(E=0)), (INV, dict(H=0)), (INV, dict(F=0)), (INV, dict(gu=None)),
    (INV, dict(dn=None)), (INV, dict(x=None)), (INV, dict(offsets=None)), (INV, dict(y=None)),
    (INV, dict(x=P + 8)), (INV, dict(y=P + 8)), (INV, dict(gu=P + 2)), (INV, dict(dn=P + 2)), (INV, dict(ws=P + 8)),
    (INV, dict(offsets=P + 2)),
    (SHAPE, dict(H=32)), (SHAPE, dict(F=96)), (SHAPE, dict(E=1025)),
    (WS, dict(ws=None)), (WS, dict(ws_bytes=4 * 64 * 2 - 1)), (moe.MOE_OK, dict(rows=0)),
    (moe.MOE_OK, dict(rows=0, gu=None, dn=None, x=None, offsets=None, y=None, ws=None)),
])
def test_grouped_refusals(want, kw):
    assert grouped(**kw) == want


def test_bf16_bindings_refuse_cpu_tensors():
    bf = torch.bfloat16
    layer = moe.moe_bf16_layer(8, 128, 64, P, P)
    x, y, ws = torch.zeros(2, 128, dtype=bf), torch.zeros(2, 128, dtype=bf), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_decode_layer_bf16(layer, x, 2, y, ws, logits=torch.zeros(2, 8))
    assert ei.value.status == INV
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_ffn_grouped_prefill_bf16(layer, x, torch.zeros(9, dtype=torch.int32), y, ws)
    assert ei.value.status == INV


def test_bf16_bindings_refuse_other_sizes_types_and_strides():
    """Everything a call would read or write past: sizes and types of every tensor, and views with gaps."""
    bf = torch.bfloat16
    layer = moe.moe_bf16_layer(8, 128, 64, P, P)
    ok = dict(x=torch.zeros(2, 128, dtype=bf), y=torch.zeros(2, 128, dtype=bf), logits=torch.zeros(2, 8),
              idx=torch.zeros(2, 2, dtype=torch.int32), w=torch.zeros(2, 2))
    bad = [dict(x=torch.zeros(2, 64, dtype=bf)), dict(x=torch.zeros(2, 128)), dict(y=torch.zeros(1, 128, dtype=bf)),
           dict(y=torch.zeros(2, 256, dtype=bf)[:, :128]), dict(logits=torch.zeros(2, 7)), dict(idx=torch.zeros(2, 2).long()),
           dict(w=torch.zeros(2, 3)), dict(residual=torch.zeros(2, 64, dtype=bf)), dict(wr=torch.zeros(7, 128, dtype=bf))]
    for kw in bad:
        a = dict(ok)
        a.update(kw)
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_decode_layer_bf16(layer, a.pop("x"), 2, a.pop("y"), torch.zeros(1 << 16, dtype=torch.uint8), **a)
        assert ei.value.status == INV, kw


# CPU tensors are refused for their device, which is looked at last: the message tells which check refused a call
def refusal(call, *args, **kw):
    with pytest.raises(moe.MoeError) as ei:
        call(*args, **kw)
    assert ei.value.status == INV
    return str(ei.value)


def decode_args(**kw):
    bf = torch.bfloat16
    a = dict(layer=moe.moe_bf16_layer(9, 128, 64, P, P), x=torch.zeros(2, 128, dtype=bf), k=2,
             y=torch.zeros(2, 128, dtype=bf), ws=torch.zeros(1 << 16, dtype=torch.uint8), wr=torch.zeros(8, 128, dtype=bf),
             logits=torch.zeros(2, 8), shared=1, shared_gate=torch.zeros(128, dtype=bf),
             residual=torch.zeros(2, 128, dtype=bf), idx=torch.zeros(2, 2, dtype=torch.int32), w=torch.zeros(2, 2))
    a.update(kw)
    return a


# a tensor of the same bytes and another type, of another size, and with gaps, for each argument
def spoilt(t):
    other = {torch.bfloat16: torch.float16, torch.float32: torch.int32, torch.int32: torch.float32}[t.dtype]
    return [t.view(other), t[..., 1:].contiguous(), torch.cat([t, t]), torch.stack([t, t], -1)[..., 0]]


DECODE_TENSORS = ["x", "y", "wr", "logits", "shared_gate", "residual", "idx", "w"]


def test_decode_binding_valid_call_is_refused_for_its_device_only():
    assert "current CUDA device" in refusal(moe.moe_decode_layer_bf16, **decode_args())
    bits = {n: decode_args()[n].view(v) for n, v in (("x", torch.int16), ("y", torch.uint16), ("wr", torch.int16))}
    assert "current CUDA device" in refusal(moe.moe_decode_layer_bf16, **decode_args(**bits))


@pytest.mark.parametrize("name", DECODE_TENSORS)
@pytest.mark.parametrize("i", range(4))
def test_decode_binding_refuses_each_tensor(name, i):
    bad = spoilt(decode_args()[name])[i]
    if name == "x" and i == 1:
        assert "moe_decode_layer_bf16: x" in refusal(moe.moe_decode_layer_bf16, **decode_args(x=bad))
    else:  # (more rows of x: y is then too short for them)
        assert "another type or size" in refusal(moe.moe_decode_layer_bf16, **decode_args(**{name: bad}))


def grouped_args(**kw):
    bf = torch.bfloat16
    a = dict(layer=moe.moe_bf16_layer(8, 128, 64, P, P), x_perm=torch.zeros(4, 128, dtype=bf),
             offsets=torch.zeros(9, dtype=torch.int32), y_perm=torch.zeros(4, 128, dtype=bf),
             ws=torch.zeros(4 * 64 * 2, dtype=torch.uint8))
    a.update(kw)
    return a


@pytest.mark.parametrize("name", ["x_perm", "offsets", "y_perm"])
@pytest.mark.parametrize("i", range(4))
def test_grouped_binding_refuses_each_tensor(name, i):
    assert "current CUDA device" in refusal(moe.moe_ffn_grouped_prefill_bf16, **grouped_args())
    msg = refusal(moe.moe_ffn_grouped_prefill_bf16, **grouped_args(**{name: spoilt(grouped_args()[name])[i]}))
    assert ("grouped_prefill_bf16: x_perm" if name == "x_perm" and i == 1 else "another type or size") in msg


def test_make_bf16_layer_refusals():
    bf = torch.bfloat16
    gu, dn = torch.zeros(4, 128, 192, dtype=bf), torch.zeros(4, 192, 64, dtype=bf)
    ok = [(gu, dn), (gu.flatten(), dn.flatten()), (gu.view(torch.int16), dn.view(torch.uint16)),
          (torch.cat([gu, gu]), torch.cat([dn, dn])), (gu.view(-1, 192), dn.view(-1, 64))]
    for a, b in ok:
        assert "one CUDA device" in refusal(moe.make_bf16_layer, 4, 192, 64, a, b)
    for a, b in [(gu.half(), dn), (gu, dn.float()), (gu.transpose(1, 2), dn), (gu, dn[:, :, ::2])]:
        assert "another type, or not contiguous" in refusal(moe.make_bf16_layer, 4, 192, 64, a, b)
    for a, b in [(gu[:3], dn), (gu, dn[:3]), (gu.transpose(1, 2).contiguous(), dn), (gu, dn.transpose(1, 2).contiguous()),
                 (gu.flatten()[1:], dn), (gu.view(2, 256, 192), dn)]:
        assert "another size" in refusal(moe.make_bf16_layer, 4, 192, 64, a, b)


@pytest.mark.parametrize("name", ["x", "w", "y", "bias", "residual"])
@pytest.mark.parametrize("i", range(4))
def test_linear_binding_refuses_each_tensor(name, i):
    bf = torch.bfloat16
    a = dict(x=torch.zeros(3, 16, dtype=bf), w=torch.zeros(8, 16, dtype=bf), y=torch.zeros(3, 8, dtype=bf),
             bias=torch.zeros(8, dtype=bf), residual=torch.zeros(3, 8, dtype=bf))
    assert "current CUDA device" in refusal(moe.moe_linear, **a)
    bad = spoilt(a[name])[i]
    if i == 3 and name != "bias":  # rows may lie apart, their elements may not
        assert bad.stride(-1) == 2
    a[name] = bad
    assert "current CUDA device" not in refusal(moe.moe_linear, **a)


def test_linear_binding_refuses_sizes_past_32_bits():
    """The ABI's sizes are ints: one that only 64 bits hold must not arrive as its lower half (2^32 rows as none)."""
    bf = torch.bfloat16
    wide = lambda r, c: torch.zeros(1, 1, dtype=bf).expand(r, c)
    for n in (1 << 31, 1 << 32, (1 << 32) + 4):
        for x, w, y in (((n, 8), (8, 8), (n, 8)), ((4, 8), (n, 8), (4, n)), ((4, n), (8, n), (4, 8))):
            with pytest.raises(moe.MoeError) as ei:
                moe.moe_linear(wide(*x), wide(*w), wide(*y))
            assert ei.value.status == SHAPE, (x, w, y)


def test_make_bf16_layer_takes_gate_and_up_as_a_dimension():
    bf = torch.bfloat16
    gu, dn = torch.zeros(4, 2, 64, 192, dtype=bf), torch.zeros(4, 192, 64, dtype=bf)
    for a in (gu, gu.view(8, 64, 192).view(4, 2, 64, 192), gu.unsqueeze(0)):
        assert "one CUDA device" in refusal(moe.make_bf16_layer, 4, 192, 64, a, dn)
    for a in (gu.view(4, 4, 32, 192), gu.view(4, 2, 192, 64)):
        want = "one CUDA device" if a.shape[-1] == 192 else "another size"
        assert want in refusal(moe.make_bf16_layer, 4, 192, 64, a, dn)
    assert "another size" in refusal(moe.make_bf16_layer, 4, 192, 64, torch.zeros(4, 3, 64, 192, dtype=bf), dn)
