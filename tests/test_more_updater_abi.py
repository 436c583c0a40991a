"""The ABI calls of the norm, the linear attention and the optimizer refuse bad arguments on the host, before anything is
launched (no GPU needed)."""
import ctypes
import math

import pytest

from gaussian_splatting_rasterizer_amd import binding as b

INVALID, SMALL, UNSUP = b.GS_ERR_INVALID_ARGUMENT, b.GS_ERR_WORKSPACE_TOO_SMALL, b.GS_ERR_UNSUPPORTED


def at(i):
    """Aligned addresses that are never read, 2^40 bytes apart."""
    return (i + 1) << 40


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(b.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return b.load_library()


# ---- the norm ------------------------------------------------------------------------------------------------------

def norm_dims(**kw):
    d = dict(rows=10, width=48, dtype=b.GS_BF16, stream_dtype=b.GS_F32, weight_dtype=b.GS_BF16, scale_group=0, eps=1e-6)
    d.update(kw)
    return b.gs_norm_dims(**d)


def norm_forward(lib, d, x=at(0), residual=at(1), weight=at(2), ld_x=48, ld_r=48, y=at(3), ld_y=48, h=at(4), ld_h=48):
    i = b.gs_norm_inputs(x, residual, weight, ld_x, ld_r)
    return lib.gs_norm_forward(ctypes.byref(d), ctypes.byref(i), y, ld_y, h, ld_h, None)


def norm_forward8(lib, d, codes=at(3), ld_codes=48, scales=at(5), x=at(0), h=at(4)):
    i = b.gs_norm_inputs(x, at(1), at(2), 48, 48)
    return lib.gs_norm_forward8(ctypes.byref(d), ctypes.byref(i), codes, ld_codes, scales, h, 48, None)


def norm_backward(lib, d, h=at(0), ld_h=48, weight=at(1), dy=at(2), ld_dy=48, dh=at(3), ld_dh=48, x=at(4), residual=at(5),
                  gw=at(6), ld_x=48, ld_r=48, ws=at(7), nbytes=1 << 30):
    g = b.gs_norm_grads(x, residual, gw, ld_x, ld_r)
    return lib.gs_norm_backward(ctypes.byref(d), h, ld_h, weight, dy, ld_dy, dh, ld_dh, ctypes.byref(g), ws, nbytes, None)


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=3), INVALID), (dict(stream_dtype=b.GS_F16), INVALID), (dict(weight_dtype=b.GS_F16), INVALID),
    (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(rows=1 << 31), UNSUP), (dict(width=(1 << 20) + 1), UNSUP)])
def test_norm_dims(lib, kw, status):
    d, size = norm_dims(**kw), ctypes.c_size_t()
    assert lib.gs_norm_size(ctypes.byref(d), ctypes.byref(size)) == status
    assert norm_forward(lib, d) == status
    assert norm_forward8(lib, d) == status
    assert norm_backward(lib, d) == status
    assert "gs_norm" in b.last_error()


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), INVALID), (dict(x=at(0) + 1), INVALID), (dict(ld_x=47), INVALID), (dict(ld_x=(1 << 21) + 1), UNSUP),
    (dict(residual=at(1) + 2), INVALID), (dict(ld_r=40), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
    (dict(ld_y=1), INVALID), (dict(h=at(4) + 2), INVALID), (dict(ld_h=0), INVALID),
    (dict(h=at(0)), INVALID),                       # float32 over the 16-bit x
    (dict(y=at(0), ld_y=56), INVALID),              # over x with another row stride
    (dict(y=at(0) + 32), INVALID), (dict(h=at(1) + 4), INVALID), (dict(h=at(1), ld_h=64), INVALID),
    (dict(y=at(1)), INVALID), (dict(y=at(2)), INVALID), (dict(h=at(2)), INVALID), (dict(y=at(4)), INVALID)])
def test_norm_forward_arguments(lib, kw, status):
    assert norm_forward(lib, norm_dims(), **kw) == status


@pytest.mark.parametrize("kw, status", [
    (dict(codes=None), INVALID), (dict(ld_codes=47), INVALID), (dict(scales=None), INVALID), (dict(scales=at(5) + 2), INVALID),
    (dict(codes=at(0)), INVALID), (dict(codes=at(1)), INVALID), (dict(scales=at(3)), INVALID), (dict(scales=at(4)), INVALID),
    (dict(scales=at(2)), INVALID), (dict(scales=at(0)), INVALID)])
def test_norm_forward8_arguments(lib, kw, status):
    assert norm_forward8(lib, norm_dims(), **kw) == status


@pytest.mark.parametrize("group", [-1, 1, 16, 48, 256])
def test_norm_scale_groups(lib, group):
    assert norm_forward8(lib, norm_dims(scale_group=group)) == INVALID


@pytest.mark.parametrize("kw, status", [
    (dict(h=None), INVALID), (dict(h=at(0) + 2), INVALID), (dict(ld_h=47), INVALID), (dict(weight=None), INVALID),
    (dict(dy=None), INVALID), (dict(ld_dy=4), INVALID), (dict(dh=at(3) + 1), INVALID), (dict(ld_dh=9), INVALID),
    (dict(ld_x=47), INVALID), (dict(ld_r=47), INVALID), (dict(gw=at(6) + 1), INVALID), (dict(ws=None), INVALID),
    (dict(ws=at(7) + 16), INVALID), (dict(nbytes=16), SMALL),
    (dict(x=at(0)), INVALID), (dict(residual=at(0)), INVALID), (dict(x=at(1)), INVALID), (dict(gw=at(1)), INVALID),
    (dict(x=at(2), ld_x=56), INVALID), (dict(residual=at(2)), INVALID), (dict(residual=at(3), ld_r=56), INVALID),
    (dict(x=at(3)), INVALID),                       # 16 bits over a float32 gradient that the same row's end still needs
    (dict(x=at(5)), INVALID), (dict(gw=at(4)), INVALID), (dict(gw=at(2)), INVALID)])
def test_norm_backward_arguments(lib, kw, status):
    assert norm_backward(lib, norm_dims(), **kw) == status


def test_norm_gradients_in_place_of_long_rows(lib):
    """Their weight gradient reads dy and h once more."""
    d = norm_dims(width=10000)
    ld = dict(ld_h=10000, ld_dy=10000, ld_dh=10000, ld_x=10000, ld_r=10000)
    assert norm_backward(lib, d, x=at(2), **ld) == INVALID


def test_norm_without_rows(lib):
    d = norm_dims(rows=0)
    assert norm_forward(lib, d, x=None, residual=None, weight=None, y=None, h=None) == b.GS_OK
    assert lib.gs_norm_forward(ctypes.byref(d), None, None, 0, None, 0, None) == INVALID
    assert lib.gs_norm_forward(None, None, None, 0, None, 0, None) == INVALID
    assert lib.gs_norm_size(ctypes.byref(norm_dims()), None) == INVALID
    assert lib.gs_norm_backward(ctypes.byref(d), None, 0, None, None, 0, None, 0, None, None, 0, None) == INVALID


# ---- linear attention ----------------------------------------------------------------------------------------------

def attn_dims(**kw):
    d = dict(rows=300, n_seq=1, heads=4, kv_heads=2, d_key=16, d_value=24, dtype=b.GS_BF16, gate_dtype=b.GS_F32,
             gate_per_row=1, scale=0.25)
    d.update(kw)
    return b.gs_attn_dims(**d)


def heads(i, count, width, **kw):
    d = dict(p=at(i), ld_row=count * width, ld_head=width)
    d.update(kw)
    return b.gs_heads(**d)


def attn_inputs(q={}, k={}, v={}, gate=at(3), ld_gate=2, state=at(4)):
    return b.gs_attn_inputs(heads(0, 4, 16, **q), heads(1, 2, 16, **k), heads(2, 2, 24, **v), gate, ld_gate, state)


def attn_forward(lib, d, inputs=None, off=None, y={}, last=at(6), saved=at(7), ws=at(8), nbytes=1 << 34):
    i, o = inputs if inputs is not None else attn_inputs(), heads(5, 4, 24, **y)
    return lib.gs_attn_forward(ctypes.byref(d), off, ctypes.byref(i), ctypes.byref(o), last, saved, ws, nbytes, None)


def attn_backward(lib, d, inputs=None, off=None, saved=at(7), dy={}, d_last=at(9), q={}, k={}, v={}, gate=at(13), ld_gate=2,
                  state=at(14), ws=at(8), nbytes=1 << 34):
    i, y = inputs if inputs is not None else attn_inputs(), heads(5, 4, 24, **dy)
    g = b.gs_attn_grads(heads(10, 4, 16, **q), heads(11, 2, 16, **k), heads(12, 2, 24, **v), gate, ld_gate, state)
    return lib.gs_attn_backward(ctypes.byref(d), off, ctypes.byref(i), saved, ctypes.byref(y), d_last, ctypes.byref(g), ws,
                                nbytes, None)


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=3), INVALID), (dict(gate_dtype=b.GS_F16), INVALID), (dict(gate_per_row=2), INVALID),
    (dict(rows=-1), INVALID), (dict(n_seq=-1), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(kv_heads=3), INVALID), (dict(heads=2, kv_heads=4), INVALID), (dict(d_key=0), INVALID), (dict(d_value=0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(rows=1 << 31), UNSUP),
    (dict(n_seq=1 << 31), UNSUP), (dict(heads=65536), UNSUP), (dict(d_key=129), UNSUP), (dict(d_value=129), UNSUP)])
def test_attn_dims(lib, kw, status):
    d = attn_dims(**kw)
    assert lib.gs_attn_sizes(ctypes.byref(d), None, None, None) == status
    assert attn_forward(lib, d) == status
    assert attn_backward(lib, d) == status
    assert "gs_attn" in b.last_error()


BAD_HEADS = [
    (dict(p=None), INVALID), (dict(p=at(0) + 1), INVALID), (dict(ld_row=-64), INVALID), (dict(ld_head=-16), INVALID),
    (dict(ld_row=1 << 24), UNSUP), (dict(ld_head=(1 << 40) + 1), UNSUP)]


@pytest.mark.parametrize("kw, status", BAD_HEADS)
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_attn_inputs(lib, name, kw, status):
    i = attn_inputs(**{name: kw})
    assert attn_forward(lib, attn_dims(), i) == status
    assert attn_backward(lib, attn_dims(), i) == status


# rows that meet rows, heads that meet heads, heads that meet the rows behind theirs
OVERLAPS = [(dict(ld_row=0), INVALID), (dict(ld_head=0), INVALID), (dict(ld_row=8), INVALID), (dict(ld_head=8), INVALID),
            (dict(ld_row=128, ld_head=128), INVALID)]


@pytest.mark.parametrize("kw, status", BAD_HEADS + OVERLAPS)
def test_attn_outputs(lib, kw, status):
    assert attn_forward(lib, attn_dims(), y=kw) == status
    if "p" not in kw or kw["p"]:
        for name in ("q", "k", "v"):
            wide = dict(kw, ld_head=kw.get("ld_head", 24)) if name == "v" else kw
            assert attn_backward(lib, attn_dims(), **{name: wide}) == status
    if (kw, status) in BAD_HEADS:
        assert attn_backward(lib, attn_dims(), dy=kw) == status


@pytest.mark.parametrize("kw, status", [
    (dict(inputs=attn_inputs(gate=None)), INVALID), (dict(inputs=attn_inputs(gate=at(3) + 2)), INVALID),
    (dict(inputs=attn_inputs(ld_gate=1)), INVALID), (dict(inputs=attn_inputs(ld_gate=(1 << 21) + 1)), UNSUP),
    (dict(inputs=attn_inputs(state=at(4) + 2)), INVALID), (dict(off=at(20) + 4), INVALID)])
def test_attn_gate_state_and_offsets(lib, kw, status):
    assert attn_forward(lib, attn_dims(), **kw) == status
    assert attn_backward(lib, attn_dims(), **kw) == status


def test_attn_sequences_of_equal_length(lib):
    assert attn_forward(lib, attn_dims(n_seq=7)) == INVALID  # 300 rows
    assert attn_forward(lib, attn_dims(n_seq=0)) == INVALID


@pytest.mark.parametrize("kw, status", [
    (dict(last=at(6) + 1), INVALID), (dict(saved=at(7) + 64), INVALID), (dict(ws=None), INVALID), (dict(ws=at(8) + 128), INVALID),
    (dict(nbytes=64), SMALL), (dict(last=at(4) + 4), INVALID), (dict(last=at(4) - 4), INVALID)])
def test_attn_forward_arguments(lib, kw, status):
    assert attn_forward(lib, attn_dims(rows=30000), **kw) == status


@pytest.mark.parametrize("kw, status", [
    (dict(saved=None), INVALID), (dict(saved=at(7) + 64), INVALID), (dict(d_last=at(9) + 2), INVALID),
    (dict(gate=at(13) + 2), INVALID), (dict(ld_gate=1), INVALID), (dict(state=at(14) + 1), INVALID),
    (dict(state=at(9) + 4), INVALID), (dict(state=at(4) + 4), INVALID), (dict(ws=None), INVALID), (dict(nbytes=64), SMALL)])
def test_attn_backward_arguments(lib, kw, status):
    assert attn_backward(lib, attn_dims(rows=30000), **kw) == status


def test_attn_null_arguments(lib):
    d, i = attn_dims(), attn_inputs()
    assert lib.gs_attn_sizes(None, None, None, None) == INVALID
    assert lib.gs_attn_forward(None, None, None, None, None, None, None, 0, None) == INVALID
    assert lib.gs_attn_forward(ctypes.byref(d), None, None, None, None, None, None, 0, None) == INVALID
    assert lib.gs_attn_forward(ctypes.byref(d), None, ctypes.byref(i), None, None, None, None, 0, None) == INVALID
    assert lib.gs_attn_backward(ctypes.byref(d), None, ctypes.byref(i), None, None, None, None, None, 0, None) == INVALID


def test_attn_sizes_grow_with_the_rows(lib):
    small, large = b.gs_attn_sizes(attn_dims(rows=20000)), b.gs_attn_sizes(attn_dims(rows=200000))
    assert all(s < l for s, l in zip(small, large))


# ---- the optimizer -------------------------------------------------------------------------------------------------

def adamw(lib, tensors, n=None, bits=32, beta1=0.9, beta2=0.999, eps=1e-8, steps=at(30), grad_scale=None, rate_scale=None,
          array=True):
    d = b.gs_adamw_dims(len(tensors) if n is None else n, bits, beta1, beta2, eps)
    a = (b.gs_adamw_tensor * max(len(tensors), 1))(*tensors)
    return lib.gs_adamw_step(ctypes.byref(d), a if array else None, steps, grad_scale, rate_scale, None)


def tensor(first=0, **kw):
    d = dict(param=at(first), grad=at(first + 1), m=at(first + 2), v=at(first + 3), m_scale=at(first + 4),
             v_scale=at(first + 5), copy=at(first + 6), n=1000, lr=1e-3, weight_decay=0.01, dtype=b.GS_F32,
             grad_dtype=b.GS_BF16, copy_dtype=b.GS_BF16)
    d.update(kw)
    return b.gs_adamw_tensor(**d)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), INVALID), (dict(array=False), INVALID), (dict(bits=16), INVALID), (dict(bits=0), INVALID),
    (dict(beta1=1.0), INVALID), (dict(beta1=-0.1), INVALID), (dict(beta2=math.nan), INVALID), (dict(beta2=1.5), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=1e-60), INVALID), (dict(eps=math.inf), INVALID), (dict(steps=None), INVALID),
    (dict(steps=at(30) + 4), INVALID), (dict(grad_scale=at(31) + 2), INVALID), (dict(rate_scale=at(31) + 1), INVALID)])
def test_adamw_arguments(lib, kw, status):
    assert adamw(lib, [tensor()], **kw) == status
    assert "gs_adamw_step" in b.last_error()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), INVALID), (dict(n=(1 << 40) + 1), UNSUP), (dict(dtype=3), INVALID), (dict(grad_dtype=-1), INVALID),
    (dict(copy_dtype=7), INVALID), (dict(lr=math.nan), INVALID), (dict(weight_decay=math.inf), INVALID),
    (dict(param=None), INVALID), (dict(param=at(0) + 2), INVALID), (dict(grad=at(1) + 1), INVALID), (dict(m=None), INVALID),
    (dict(v=None), INVALID), (dict(copy=at(6) + 1), INVALID),
    (dict(m=at(0)), INVALID), (dict(v=at(2)), INVALID), (dict(copy=at(0)), INVALID), (dict(grad=at(0)), INVALID),
    (dict(grad=at(2) + 2), INVALID), (dict(grad=at(0) + 3998), INVALID), (dict(copy=at(1)), INVALID),
    (dict(copy=at(30)), INVALID), (dict(grad=at(30) + 8), INVALID)])
def test_adamw_tensors(lib, bits, kw, status):
    assert adamw(lib, [tensor(first=10), tensor(**kw)], bits=bits) == status


@pytest.mark.parametrize("kw, status", [
    (dict(m_scale=None), INVALID), (dict(v_scale=None), INVALID), (dict(m_scale=at(4) + 2), INVALID),
    (dict(v_scale=at(4)), INVALID), (dict(m_scale=at(2)), INVALID), (dict(v_scale=at(1)), INVALID)])
def test_adamw_scales(lib, kw, status):
    assert adamw(lib, [tensor(**kw)], bits=8) == status


def test_adamw_tensors_of_two_entries(lib):
    """The same tensor twice, a part of another's, and a state that two share."""
    for kw in (dict(param=at(0)), dict(param=at(0) + 400), dict(m=at(2)), dict(v=at(0)), dict(grad=at(0)), dict(copy=at(0))):
        assert adamw(lib, [tensor(), tensor(first=10, **kw)]) == INVALID
    many = [tensor(first=10 * i) for i in range(50)]
    assert adamw(lib, many + [tensor(first=600, v=at(203) + 3996)], steps=at(900)) == INVALID
    assert adamw(lib, [tensor(n=1 << 40), tensor(first=10, n=1)]) == UNSUP
    assert lib.gs_adamw_step(None, None, at(0), None, None, None) == INVALID
