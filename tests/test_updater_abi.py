"""The updater's ABI calls refuse bad arguments on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest

from gaussian_splatting_rasterizer_amd import binding as b

PTR = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(b.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return b.load_library()


def ffn_dims(**kw):
    d = dict(rows=10, d_in=16, d_hidden=32, d_out=8, dtype=b.GS_BF16, activation=b.GS_ACT_SILU)
    d.update(kw)
    return b.gs_ffn_dims(*[d[k] for k in ("rows", "d_in", "d_hidden", "d_out", "dtype", "activation")])


def ffn_forward(lib, d, x=PTR, ldx=16, w=(PTR, PTR, PTR), y=PTR, ldy=8, saved=None, ws=PTR, nbytes=1 << 30):
    return lib.gs_ffn_forward(ctypes.byref(d), x, ldx, ctypes.byref(b.gs_ffn_weights(*w)), y, ldy, saved, ws, nbytes,
                              None)


INVALID, SMALL, UNSUP = b.GS_ERR_INVALID_ARGUMENT, b.GS_ERR_WORKSPACE_TOO_SMALL, b.GS_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(activation=2), INVALID), (dict(rows=-1), INVALID),
    (dict(d_in=0), INVALID), (dict(d_hidden=0), INVALID), (dict(d_out=-4), INVALID), (dict(rows=1 << 31), UNSUP),
    (dict(d_hidden=(1 << 20) + 1), UNSUP)])
def test_ffn_dims(lib, kw, status):
    d = ffn_dims(**kw)
    assert lib.gs_ffn_sizes(ctypes.byref(d), None, None, None) == status
    assert ffn_forward(lib, d) == status
    assert "gs_ffn" in b.last_error()


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), INVALID), (dict(x=PTR + 1), INVALID), (dict(ldx=15), INVALID), (dict(ldx=(1 << 21) + 1), UNSUP),
    (dict(y=None), INVALID), (dict(ldy=7), INVALID), (dict(w=(None, PTR, PTR)), INVALID),
    (dict(w=(PTR, PTR + 1, PTR)), INVALID), (dict(w=(PTR, PTR, None)), INVALID), (dict(ws=None), INVALID),
    (dict(ws=PTR + 128), INVALID), (dict(nbytes=64), SMALL), (dict(saved=PTR + 16), INVALID)])
def test_ffn_forward_arguments(lib, kw, status):
    assert ffn_forward(lib, ffn_dims(), **kw) == status


def test_ffn_backward_arguments(lib):
    d, w = ffn_dims(), b.gs_ffn_weights(PTR, PTR, PTR)

    def call(saved=PTR, dy=PTR, lddy=8, grads=b.gs_ffn_grads(PTR, 16, PTR, PTR, PTR), ws=PTR, nbytes=1 << 30):
        return lib.gs_ffn_backward(ctypes.byref(d), PTR, 16, ctypes.byref(w), saved, dy, lddy,
                                   ctypes.byref(grads) if grads is not None else None, ws, nbytes, None)

    assert call(saved=None) == INVALID
    assert call(saved=PTR + 64) == INVALID
    assert call(dy=None) == INVALID
    assert call(lddy=4) == INVALID
    assert call(grads=None) == INVALID
    assert call(grads=b.gs_ffn_grads(PTR, 8, PTR, PTR, PTR)) == INVALID
    assert call(grads=b.gs_ffn_grads(PTR, 16, PTR + 1, PTR, PTR)) == INVALID
    assert call(nbytes=256) == SMALL
    assert lib.gs_ffn_backward(None, PTR, 16, ctypes.byref(w), PTR, PTR, 8, None, PTR, 1, None) == INVALID


def test_ffn_sizes_grow_with_the_rows(lib):
    small, large = b.gs_ffn_sizes(ffn_dims(rows=100)), b.gs_ffn_sizes(ffn_dims(rows=10000))
    assert all(s < l for s, l in zip(small, large))
    assert b.gs_ffn_sizes(ffn_dims(dtype=b.GS_F32))[0] > b.gs_ffn_sizes(ffn_dims())[0]
    assert ffn_forward(lib, ffn_dims(rows=0), x=None, y=None, ws=None, nbytes=0) == b.GS_OK  # nothing to do


def scan_dims(**kw):
    d = dict(rows=12, n_seq=3, channels=8, dtype=b.GS_F32)
    d.update(kw)
    return b.gs_scan_dims(d["rows"], d["n_seq"], d["channels"], d["dtype"])


def scan_forward(lib, d, off=None, inp=(PTR, PTR, PTR, 8, 8), y=PTR, ldy=8, h_last=PTR, saved=None, ws=PTR,
                 nbytes=1 << 20):
    i = b.gs_scan_inputs(*inp)
    return lib.gs_scan_forward(ctypes.byref(d), off, ctypes.byref(i), y, ldy, h_last, saved, ws, nbytes, None)


@pytest.mark.parametrize("kw, status", [
    (dict(rows=-1), INVALID), (dict(n_seq=-1), INVALID), (dict(channels=0), INVALID), (dict(dtype=7), INVALID),
    (dict(rows=1 << 31), UNSUP), (dict(channels=(1 << 20) + 1), UNSUP), (dict(rows=13), INVALID),
    (dict(n_seq=0), INVALID)])
def test_scan_dims(lib, kw, status):
    assert scan_forward(lib, scan_dims(**kw)) == status


@pytest.mark.parametrize("kw, status", [
    (dict(inp=(None, PTR, None, 8, 8)), INVALID), (dict(inp=(PTR, PTR + 2, None, 8, 8)), INVALID),
    (dict(inp=(PTR, PTR, PTR + 1, 8, 8)), INVALID), (dict(inp=(PTR, PTR, None, 7, 8)), INVALID),
    (dict(inp=(PTR, PTR, None, 8, (1 << 21) + 8)), UNSUP), (dict(off=PTR + 4), INVALID), (dict(y=None), INVALID),
    (dict(ldy=4), INVALID), (dict(h_last=PTR + 2), INVALID), (dict(saved=PTR + 8), INVALID), (dict(ws=None), INVALID),
    (dict(nbytes=8), SMALL)])
def test_scan_forward_arguments(lib, kw, status):
    assert scan_forward(lib, scan_dims(), **kw) == status


def test_scan_backward_arguments(lib):
    d, i = scan_dims(), b.gs_scan_inputs(PTR, PTR, None, 8, 8)

    def call(saved=PTR, dy=PTR, lddy=8, dhl=None, grads=b.gs_scan_grads(PTR, PTR, None, 8, 8), nbytes=1 << 20):
        return lib.gs_scan_backward(ctypes.byref(d), None, ctypes.byref(i), saved, dy, lddy, dhl,
                                    ctypes.byref(grads) if grads is not None else None, PTR, nbytes, None)

    assert call(saved=None) == INVALID
    assert call(dy=None) == INVALID
    assert call(lddy=3) == INVALID
    assert call(dhl=PTR + 1) == INVALID
    assert call(grads=None) == INVALID
    assert call(grads=b.gs_scan_grads(PTR, PTR, None, 4, 8)) == INVALID
    assert call(nbytes=16) == SMALL


def test_scan_states_in_place(lib):
    """h_last may be h0 (and dh0 dh_last or h0), but no other overlap: 3 sequences of 8 channels are 96 bytes."""
    for shift in (-92, -32, 4, 92):
        assert scan_forward(lib, scan_dims(), h_last=PTR + shift) == INVALID
        assert "overlaps" in b.last_error()
        i, g = b.gs_scan_inputs(PTR, PTR, PTR, 8, 8), b.gs_scan_grads(PTR, PTR, PTR + shift, 8, 8)
        for h0, dhl in ((PTR, None), (None, PTR)):
            i.h0 = h0
            assert lib.gs_scan_backward(ctypes.byref(scan_dims()), None, ctypes.byref(i), PTR, PTR, 8, dhl,
                                        ctypes.byref(g), PTR, 1 << 20, None) == INVALID
            assert "overlaps" in b.last_error()
    # the same array and neighbouring ones get as far as the workspace
    for h_last in (PTR, PTR + 96, PTR - 96):
        assert scan_forward(lib, scan_dims(), h_last=h_last, nbytes=8) == SMALL


def ortho_dims(**kw):
    d = b.gs_default_ortho_dims()
    for k, v in dict(dict(rows=200, cols=300, batch=2, dtype=b.GS_F32, out_dtype=b.GS_BF16), **kw).items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw, status", [
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(batch=-1), INVALID), (dict(steps=0), INVALID),
    (dict(dtype=b.GS_F16), INVALID), (dict(out_dtype=9), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(steps=65), UNSUP), (dict(rows=40000, cols=40000), UNSUP),
    (dict(cols=(1 << 20) + 1), UNSUP), (dict(batch=65536), UNSUP)])
def test_ortho_dims(lib, kw, status):
    d = ortho_dims(**kw)
    out = ctypes.c_size_t(0)
    assert lib.gs_ortho_size(ctypes.byref(d), ctypes.byref(out)) == status
    assert lib.gs_orthogonalize(ctypes.byref(d), PTR, PTR, PTR, 1 << 40, None) == status


@pytest.mark.parametrize("coef, steps, status", [
    ((1.5, -0.5, 0.0), 64, b.GS_OK), ((3.4445, -4.7750, 2.0315), 64, b.GS_OK), ((1.875, -1.25, 0.375), 64, b.GS_OK),
    ((3.0, -0.1, 0.0), 2, b.GS_OK),                   # s reaches 6.3, s^2 before the last step 8.4
    ((8.2872, -23.5959, 17.3004), 1, b.GS_OK),        # |b s^2 + c s^4| reaches 8.05
    ((8.2872, -23.5959, 17.3004), 5, UNSUP),          # s reaches 2, then 370
    ((15.0, 0.0, 0.0), 2, b.GS_OK), ((15.0, 0.0, 0.0), 3, UNSUP),  # s = 15, 225, 3375
    ((0.0, 0.0, 300.0), 1, UNSUP), ((1.0, 300.0, 0.0), 1, UNSUP), ((0.0, 0.0, 0.0), 3, b.GS_OK),
    ((float("nan"), 0.0, 0.0), 1, INVALID), ((1.0, float("inf"), 0.0), 1, INVALID),
    ((1.0, 0.0, float("-inf")), 1, INVALID)])
@pytest.mark.parametrize("shape", [(64, 128), (200, 300)], ids=str)
def test_ortho_coefficients(lib, shape, coef, steps, status):
    """Accepted where X, P and Q stay in range, refused before anything is launched otherwise."""
    d = ortho_dims(rows=shape[0], cols=shape[1], a=coef[0], b=coef[1], c=coef[2], steps=steps)
    out = ctypes.c_size_t(0)
    assert lib.gs_ortho_size(ctypes.byref(d), ctypes.byref(out)) == status
    if status != b.GS_OK:
        assert lib.gs_orthogonalize(ctypes.byref(d), PTR, PTR, PTR, 1 << 40, None) == status


def test_ortho_arguments(lib):
    d = ortho_dims()
    assert lib.gs_orthogonalize(ctypes.byref(d), None, PTR, PTR, 1 << 30, None) == INVALID
    assert lib.gs_orthogonalize(ctypes.byref(d), PTR + 2, PTR, PTR, 1 << 30, None) == INVALID
    assert lib.gs_orthogonalize(ctypes.byref(d), PTR, None, PTR, 1 << 30, None) == INVALID
    assert lib.gs_orthogonalize(ctypes.byref(d), PTR, PTR, None, 1 << 30, None) == INVALID
    assert lib.gs_orthogonalize(ctypes.byref(d), PTR, PTR, PTR, 256, None) == SMALL
    assert "needs" in b.last_error()
    d = ortho_dims(batch=0)
    assert lib.gs_orthogonalize(ctypes.byref(d), None, None, None, 0, None) == b.GS_OK
    assert b.gs_default_ortho_dims().steps == 5
