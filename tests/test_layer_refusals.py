"""CPU: what the norms, router, expert layer and 4-bit linear refuse, at the C
ABI (addresses that are never read) and in the Python binding."""
import ctypes
import os

import pytest
import torch

import block_scaled_fp8_fp8blk_amd as fb

P = 1 << 24  # a fake, aligned address: every call here refuses before any device work
S = 1 << 24  # distance between fake buffers


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fb.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fb.load()


def _norm(lib, **kw):
    a = dict(resid=P, kind=0, y=P + S, N=4, cols=64, post=P + 2 * S, gate=P + 3 * S, gate_rows=1, scale=1.0,
             out=P + 4 * S, pre=P + 5 * S, eps=1e-6, x=P + 6 * S)
    a.update(kw)
    return lib.fp8blk_block_norm(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(N=0), dict(N=fb.MAX_PANEL + 1), dict(cols=8), dict(cols=24), dict(cols=65552), dict(kind=2), dict(kind=-1),
    dict(resid=None), dict(out=None), dict(pre=None), dict(x=None), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(gate_rows=0), dict(gate_rows=2), dict(gate=None), dict(y=None),
    dict(y=None, out=None), dict(y=None, out=None, post=None), dict(y=None, out=None, post=None, gate=None),
    dict(y=None, out=None, post=None, gate=None, gate_rows=0, pre=None, x=None),
    dict(resid=P + 8), dict(y=P + S + 4), dict(post=P + 2 * S + 2), dict(gate=P + 8), dict(out=P + 4 * S + 8),
    dict(pre=P + 2), dict(x=P + 6 * S + 2),
    # outputs over inputs or each other; resid_out may be resid itself and no other part of it
    dict(out=P + 256), dict(out=P - 256), dict(out=P + S), dict(out=P + 2 * S), dict(out=P + 3 * S), dict(out=P + 5 * S),
    dict(out=P + 6 * S), dict(out=P + 6 * S + 496), dict(x=P), dict(x=P + S), dict(x=P + 2 * S + 112), dict(x=P + 3 * S),
    dict(x=P + 5 * S), dict(x=P + 4 * S + 1008)])
def test_norm_refusals(lib, kw):
    assert _norm(lib, **kw) == fb.ERR_ARG


def _route(lib, **kw):
    a = dict(w=P, bias=P, E=16, cols=64, x=P, M=2, score=0, K=4, norm=1, scale=1.0, ids=P, p=P, ws=P, wsb=1 << 20)
    a.update(kw)
    return lib.fp8blk_moe_route(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(E=0), dict(E=fb.MAX_EXPERTS + 1), dict(cols=8), dict(cols=40), dict(cols=65552), dict(M=0),
    dict(M=fb.MAX_PANEL + 1), dict(score=-1), dict(score=3), dict(K=0), dict(K=17, E=64), dict(K=5, E=4), dict(w=None),
    dict(x=None), dict(ids=None), dict(p=None), dict(w=P + 8), dict(x=P + 2), dict(bias=P + 2), dict(ids=P + 1),
    dict(p=P + 2)])
def test_route_refusals(lib, kw):
    assert _route(lib, **kw) == fb.ERR_ARG


def test_route_workspace(lib):
    need = fb.fp8blk_workspace_bytes(fb.OP_MOE_ROUTE, 16, 64, 2)
    assert need > 0 and need % 256 == 0
    assert _route(lib, ws=None) == fb.ERR_WORKSPACE
    assert _route(lib, ws=P + 64) == fb.ERR_WORKSPACE
    assert _route(lib, wsb=need - 1) == fb.ERR_WORKSPACE
    for bad in ((0, 64, 2), (1025, 64, 2), (16, 8, 2), (16, 64, 0), (16, 64, fb.MAX_PANEL + 1)):
        assert fb.fp8blk_workspace_bytes(fb.OP_MOE_ROUTE, *bad) == 0


def _moe(lib, layer=None, **kw):
    f = dict(gate=P, gate_scales=P, up=P, up_scales=P, down=P, down_scales=P, gate_global=P, up_global=P, down_global=P,
             experts=8, hidden=64, inter=96, fmt=fb.FMT_NVFP4, limit=0.0)
    f.update(layer or {})
    a = dict(layer=ctypes.byref(fb.Fp4MoeLayer(**f)), x=P, M=2, ids=P, p=P, K=3, base=P, y=P + S, ws=P, wsb=1 << 20)
    a.update(kw)
    return lib.fp4_moe(*a.values(), None)


@pytest.mark.parametrize("layer", [
    dict(fmt=2), dict(fmt=-1), dict(experts=0), dict(experts=fb.MAX_EXPERTS + 1), dict(hidden=16), dict(hidden=80),
    dict(hidden=65568), dict(inter=0), dict(inter=48), dict(inter=fb.MAX_INTER + 32), dict(limit=-1.0), dict(limit=float("inf")),
    dict(limit=float("nan")), dict(gate=None), dict(up_scales=None), dict(down=None), dict(gate=P + 8), dict(up=P + 4),
    dict(down_scales=P + 4), dict(gate_scales=P + 2), dict(fmt=fb.FMT_MXFP4, up_scales=P + 2), dict(gate_global=P + 2)])
def test_moe_layer_refusals(lib, layer):
    assert _moe(lib, layer) == fb.ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(M=0), dict(M=17), dict(K=0), dict(K=17), dict(x=None), dict(ids=None), dict(p=None),
    dict(y=None), dict(x=P + 8), dict(y=P + S + 4), dict(ids=P + 2), dict(p=P + 1), dict(base=P + 4),
    # y over x, ids, weights, or part of base
    dict(y=P + 128), dict(x=P + S, y=P + S), dict(ids=P + S + 8, x=P), dict(p=P + S + 504), dict(base=P + S + 256),
    dict(base=P + S - 256)])
def test_moe_refusals(lib, kw):
    assert _moe(lib, **kw) == fb.ERR_ARG


def test_moe_workspace(lib):
    assert lib.fp4_moe(None, P, 2, P, P, 3, P, P + S, P, 1 << 20, None) == fb.ERR_ARG
    need = fb.fp4_moe_bytes(96, 2, 3)
    assert need > 0 and need % 256 == 0
    assert _moe(lib, ws=None) == fb.ERR_WORKSPACE
    assert _moe(lib, ws=P + 128) == fb.ERR_WORKSPACE
    assert _moe(lib, wsb=need - 1) == fb.ERR_WORKSPACE
    for bad in ((16, 1, 1), (48, 1, 1), (fb.MAX_INTER + 32, 1, 1), (64, 0, 1), (64, 17, 1), (64, 1, 0), (64, 1, 17)):
        assert fb.fp4_moe_bytes(*bad) == 0


@pytest.mark.parametrize("kw", [
    dict(group=16), dict(group=0), dict(group=256), dict(rows=0), dict(rows=-3), dict(cols=16), dict(cols=48),
    dict(cols=96, group=64), dict(cols=192, group=128), dict(cols=65568), dict(M=0), dict(M=17), dict(codes=None),
    dict(scales=None), dict(x=None), dict(y=None), dict(codes=P + 8), dict(scales=P + 1), dict(x=P + 2), dict(y=P + 2)])
def test_int4_refusals(lib, kw):
    a = dict(codes=P, scales=P, zeros=P, group=32, rows=4, cols=64, x=P, M=1, y=P + S)
    a.update(kw)
    assert lib.int4_gemv(*a.values(), None) == fb.ERR_ARG


def test_binding_refuses_host_tensors(lib):
    t = torch.zeros(2, 32)
    for call in (lambda: fb.fp8blk_block_norm(t, None, None, None, 1.0, None, t[0], 1e-6, t),
                 lambda: fb.fp8blk_moe_route(t, None, t, 0, True, 1.0, t, t, None),
                 lambda: fb.fp4_moe_weights(0, *[t] * 9), lambda: fb.int4_gemv(t, t, None, 32, t, t)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="FMT"):
        fb.fp4_moe_weights(2, *[t] * 9)


class _Gpu0:
    """Stands in for a tensor on GPU 0 where there is none: what the binding's checks read."""

    def __init__(self, shape, dtype, device=0, contiguous=True):
        self.shape, self.dtype, self._d, self._c = torch.Size(shape), dtype, device, contiguous
        self.device = f"cuda:{device}"

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self._d

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return P


def test_binding_checks_a_buffer():
    t = _Gpu0((2, 32), torch.float32)
    f32 = (torch.float32,)
    assert fb._buf(None, 0, f32, (2, 32), "t", False) is None and fb._buf(t, 0, f32, (2, 32), "t") == P
    with pytest.raises(ValueError, match="needed"):
        fb._buf(None, 0, f32, (2, 32), "t")
    with pytest.raises(ValueError, match="device 1"):
        fb._buf(t, 1, f32, (2, 32), "t")
    with pytest.raises(TypeError, match="dtype"):
        fb._buf(t, 0, (torch.uint8,), (2, 32), "t")
    with pytest.raises(ValueError, match="shape"):
        fb._buf(t, 0, f32, (32, 2), "t")
    with pytest.raises(ValueError, match="contiguous"):
        fb._buf(_Gpu0((2, 32), torch.float32, contiguous=False), 0, f32, (2, 32), "t")
