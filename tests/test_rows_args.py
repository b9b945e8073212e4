"""Refusals of the operators on rows of logits, on the host (no GPU call is made)."""
import ctypes as C

import pytest

from block_diffusion_draft_dflash_gb300 import _lib

A = 1 << 20            # an aligned address that nothing reads


def rows(data=A, dtype=0, n=4, V=100, ld=None):
    return _lib.RowsStruct(data, dtype, n, V, V if ld is None else ld)


def sample(x=None, group=1, u=A, token=A, ws=A, ws_bytes=512):
    x = rows() if x is None else x
    return _lib.load().dflash_sample(C.addressof(x), group, None, None, None, None, u, token, None, None, ws, ws_bytes, None)


def top(x=None, K=5, T=1.0, id=A, val=A, ws=A, ws_bytes=512):
    x = rows() if x is None else x
    return _lib.load().dflash_top_logits(C.addressof(x), K, T, id, val, None, ws, ws_bytes, None)


def distill(x=None, K=5, lists=4, id=A, val=A, row=None, T=1.0, loss=A, stats=A, grad=None, ld=100, ws=A, ws_bytes=512):
    x = rows() if x is None else x
    return _lib.load().dflash_distill(C.addressof(x), K, lists, id, val, None, row, T, None, loss, stats, grad, ld, ws, ws_bytes, None)


def backward(x=None, K=5, lists=4, id=A, val=A, row=None, T=1.0, stats=A, grad=2 * A, ld=100, ws=A, ws_bytes=512):
    x = rows() if x is None else x
    return _lib.load().dflash_distill_backward(C.addressof(x), K, lists, id, val, None, row, T, None, stats, None, grad, ld, ws, ws_bytes, None)


BAD_ROWS = [(dict(n=-1), -1), (dict(V=0), -1), (dict(dtype=2), -1), (dict(dtype=-1), -1), (dict(ld=99), -1), (dict(data=None), -1),
            (dict(data=A + 4), -3), (dict(V=(1 << 20) + 1), -2), (dict(n=(1 << 27) + 1), -2), (dict(ld=1 << 61), -2)]


@pytest.mark.parametrize("call", [sample, top, distill, backward])
@pytest.mark.parametrize("bad,code", BAD_ROWS)
def test_rows(call, bad, code):
    assert call(rows(**bad), **({"lists": 1 << 28, "ld": 1 << 20} if call in (distill, backward) else {})) == code


@pytest.mark.parametrize("call", [sample, top, distill, backward])
def test_workspace_and_no_rows(call):
    assert call(ws=None) == -9 and call(ws_bytes=128) == -9
    assert call(rows(n=0, data=None)) == 0


def test_null_rows():
    lib = _lib.load()
    assert lib.dflash_sample(None, 1, *[None] * 9, 0, None) == -1
    assert lib.dflash_top_logits(None, 1, 1.0, *[None] * 4, 0, None) == -1


def test_sample():
    assert sample(group=0) == -1 and sample(group=3) == -1 and sample(u=None) == -1 and sample(token=None) == -1


def test_top():
    assert top(K=0) == -1 and top(K=1025) == -2 and top(id=None) == -1 and top(val=None) == -1
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-38, 1e38):
        assert top(T=T) == -1


@pytest.mark.parametrize("call", [distill, backward])
def test_distill(call):
    assert call(K=0) == -1 and call(K=1025) == -2 and call(lists=-1) == -1 and call(lists=3) == -1
    assert call(id=None) == -1 and call(val=None) == -1 and call(stats=None) == -1 and call(stats=A + 8) == -3
    assert call(grad=2 * A, ld=99) == -1 and call(grad=2 * A + 2) == -3 and call(grad=2 * A, ld=1 << 61) == -2
    assert call(grad=A + 16) == -1 and call(grad=A, ld=101) == -1 and call(grad=A - 16, ld=100) == -1     # half over the student's
    for T in (0.0, -1.0, float("nan"), float("inf")):
        assert call(T=T) == -1


def test_outputs():
    assert distill(loss=None) == -1 and backward(grad=None) == -1


def test_path_rows():
    lib = _lib.load()
    call = lambda b=2, D=4, n=9, new=A, src=A, ms=4, cl=A, out=A: lib.dflash_path_rows(b, D, n, new, src, ms, cl, out, None)  # noqa: E731
    assert call(b=-1) == -1 and call(D=0) == -1 and call(n=0) == -1 and call(ms=2) == -1 and call(ms=-1) == -1
    assert call(new=None) == -1 and call(src=None) == -1 and call(cl=None) == -1 and call(out=None) == -1
    assert call(b=1 << 28) == -2 and call(b=0, new=None) == 0


def test_filtered_forward():
    import synth
    from block_diffusion_draft_dflash_gb300 import engine

    m = engine.DeviceModel.from_host(synth.target_weights(synth.ModelShape(1, 128, 2, 1, 128, 128, 64), 1), "cpu")
    lib = _lib.load()
    size = lib.dflash_target_tree_forward_filtered_workspace_size(C.byref(m.cfg), 1, 3)
    assert size > lib.dflash_target_tree_forward_workspace_size(C.byref(m.cfg), 1, 3)

    def call(K=0, T=1.0, ids=A, vals=A, ws_bytes=size, ws=A):
        return lib.dflash_target_tree_forward_filtered(
            C.byref(m.cfg), C.byref(m.weights), 1, 3, A, None, None, A, A, 64, A, None, None, None, None, 0, K, T, ids, vals, None,
            A, None, ws, ws_bytes, None)
    assert call(K=-1) == -1 and call(K=1025) == -2 and call(K=4, ids=None) == -1 and call(K=4, vals=None) == -1
    assert call(K=4, T=0.0) == -1 and call(K=4, T=float("nan")) == -1
    assert call(ws=None) == -9 and call(ws_bytes=size - 256) == -9
