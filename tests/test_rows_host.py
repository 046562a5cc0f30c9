"""Refusals of the feature-row operators (embedding, RMS norm, 8-bit rows) that need no GPU:
every rejected argument returns before anything is enqueued, and the binding checks shapes,
types and devices before the library sees a pointer."""
import ctypes

import pytest
import torch

import sparse_convolution_voxel_b200 as scv
from sparse_convolution_voxel_b200 import _lib

P = ctypes.c_void_p
A, B, C = P(4096), P(8192), P(12288)   # aligned addresses that nothing dereferences
ARG, WORKSPACE = 1, 128


@pytest.fixture(scope="module")
def lib():
    from sparse_convolution_voxel_b200 import build
    build.build()
    return _lib.load()


def test_embed_argument_checks(lib):
    def fwd(ids=A, w=4, n=10, table=B, vocab=100, c=16, y=C, dt=0):
        return lib.lat_embed_fwd(ids, w, n, table, vocab, c, 1.0, -1, y, dt, None, None)

    assert fwd(ids=None) == fwd(table=None) == fwd(y=None) == ARG
    assert fwd(w=2) == fwd(n=-1) == fwd(n=1 << 31) == fwd(vocab=0) == fwd(vocab=(1 << 31) - 1) == ARG
    assert fwd(c=12) == fwd(c=0) == fwd(c=16392) == fwd(dt=3) == ARG
    assert fwd(table=P(4104)) == fwd(y=P(4104)) == fwd(ids=P(4098)) == fwd(ids=P(4100), w=8) == ARG
    assert fwd(n=0) == 0                                                       # nothing to enqueue

    def wgrad(ids=A, w=8, n=10, dy=B, vocab=100, c=16, out=C, dt=2, ws=P(1 << 20), size=1 << 30):
        return lib.lat_embed_wgrad(ids, w, n, dy, vocab, c, 1.0, -1, out, dt, ws, size, None, None)

    assert wgrad(ids=None) == wgrad(dy=None) == wgrad(out=None) == wgrad(w=1) == wgrad(c=20) == wgrad(dt=-1) == ARG
    assert wgrad(dy=P(4104)) == wgrad(out=P(4112)) == ARG
    need = lib.lat_embed_wgrad_ws_bytes(10, 100, 16)
    assert need > 0 and wgrad(size=need - 1) == wgrad(ws=None) == wgrad(ws=P(4104)) == WORKSPACE
    assert lib.lat_embed_wgrad_ws_bytes(-1, 100, 16) == lib.lat_embed_wgrad_ws_bytes(10, 0, 16) == 0
    assert lib.lat_embed_wgrad_ws_bytes(10, 100, 17) == 0


def test_q8_argument_checks(lib):
    def pack(x=A, n=10, c=40, q=B, s=C, dt=1):
        return lib.lat_q8_pack(x, n, c, q, s, dt, None)

    def unpack(x=A, n=10, c=40, q=B, s=C, dt=1):
        return lib.lat_q8_unpack(q, s, n, c, x, dt, None)

    for f in (pack, unpack):
        assert f(x=None) == f(q=None) == f(s=None) == f(n=-1) == f(c=4) == f(c=16400) == f(dt=7) == ARG
        assert f(x=P(4104)) == f(q=P(4104)) == ARG
        assert f(n=0) == 0
    km = _lib.lat_kmap()
    km.k3, km.n_out, km.n_in, km.pair_capacity = 27, 10, 10, 100
    km.nbr, km.perm, km.tile_mask, km.pair_off, km.pair_in, km.pair_out = (P(4096),) * 6

    def wgrad(q=A, s=B, cin=16, dy=C, cout=16, m=km, dw=P(16384), dt=1, ws=P(1 << 20), size=1 << 30):
        return lib.lat_sconv_wgrad_q8(q, s, cin, dy, cout, ctypes.byref(m), dw, dt, ws, size, None, None)

    assert wgrad(q=None) == wgrad(s=None) == wgrad(dw=None) == wgrad(cin=12) == wgrad(cout=264) == wgrad(dt=5) == ARG
    assert wgrad(q=P(4104)) == wgrad(dy=P(4104)) == ARG
    need = lib.lat_sconv_wgrad_q8_ws_bytes(16, 16, ctypes.byref(km), 1)
    assert need > 0 and wgrad(size=need - 1) == wgrad(ws=None) == WORKSPACE
    km.pair_in = None
    assert wgrad() == ARG


def test_norm_argument_checks(lib):
    def fwd(x=A, res=None, w=None, n=10, c=16, eps=1e-6, h=None, y=B, y8=None, y8s=None, h8=None, h8s=None, dt=0):
        return lib.lat_rms_norm_fwd(x, res, w, n, c, eps, h, y, y8, y8s, h8, h8s, None, dt, None)

    assert fwd(x=None) == fwd(n=-1) == fwd(c=10) == fwd(c=16392) == fwd(dt=9) == ARG
    assert fwd(eps=0.0) == fwd(eps=-1.0) == fwd(eps=float("nan")) == fwd(eps=float("inf")) == ARG
    assert fwd(y8=C) == fwd(y8s=C) == fwd(h8=C) == fwd(h8s=C) == ARG               # values without scales
    assert fwd(x=P(4104)) == fwd(res=P(4104)) == fwd(w=P(4104)) == fwd(y=P(4104)) == fwd(h=P(4104)) == ARG
    assert fwd(n=0) == 0

    def bwd(dy=A, dh=None, h=B, h8=None, h8s=None, rstd=C, w=None, n=10, c=16, dx=P(16384), dw=P(20480), dt=0,
            ws=P(1 << 20), size=1 << 30):
        return lib.lat_rms_norm_bwd(dy, dh, h, h8, h8s, rstd, w, n, c, dx, dw, dt, ws, size, None)

    assert bwd(dy=None) == bwd(h=None) == bwd(rstd=None) == bwd(dx=None) == bwd(c=12) == bwd(dt=4) == ARG
    assert bwd(h8=A, h8s=A) == bwd(h=None, h8=A) == ARG                            # both forms of h; no scales
    assert bwd(dy=P(4104)) == bwd(dh=P(4104)) == bwd(dw=P(4098)) == bwd(dx=P(4104)) == ARG
    need = lib.lat_rms_norm_bwd_ws_bytes(10, 16)
    assert need > 0 and bwd(size=need - 1) == bwd(ws=None) == WORKSPACE
    assert bwd(n=0, dw=None) == 0                                                   # no rows, no dw


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros(4, 16)
    ids = torch.zeros(4, dtype=torch.int32)
    q, s = torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8)
    f32 = torch.float32
    with pytest.raises(ValueError, match="device tensors"):                         # no CPU path
        scv.embed_fwd(ids, x)
    with pytest.raises(ValueError, match="device tensors"):
        scv.embed_wgrad(ids, x, 10)
    with pytest.raises(ValueError, match="device tensors"):
        scv.rms_norm_fwd(x)
    with pytest.raises(ValueError, match="device tensors"):
        scv.rms_norm_bwd(x, x, torch.zeros(4))
    with pytest.raises(ValueError, match="device tensors"):
        scv.q8_pack(x)
    with pytest.raises(ValueError, match="device tensors"):
        scv.q8_unpack(scv.Q8Rows(q, s))
    for bad in (ids.float(), ids.view(2, 2), torch.zeros(4, dtype=torch.int16), ids[:3]):
        with pytest.raises(ValueError, match="ids"):
            _lib.lat_embed_fwd(bad, x, 1.0, -1, x)
    with pytest.raises(ValueError, match="ids"):
        _lib.lat_embed_wgrad(ids[:3], x, 1.0, -1, x)
    with pytest.raises(ValueError, match="table"):
        _lib.lat_embed_fwd(ids, x.double(), 1.0, -1, x)
    for f in (lambda: scv.embed_fwd(ids, x[0]), lambda: scv.embed_fwd(ids[0], x), lambda: scv.embed_wgrad(ids, x[0], 10),
              lambda: scv.rms_norm_bwd(x[0], x[0], torch.zeros(1)), lambda: scv.rms_norm_fwd(x[0]),
              lambda: scv.q8_pack(x[None]), lambda: scv.conv_wgrad_q8(scv.Q8Rows(q, s), x[0], None)):
        with pytest.raises(ValueError):                                             # rows are (n, c), ids (n,)
            f()
    with pytest.raises(ValueError, match="dtable"):
        _lib.lat_embed_wgrad(ids, x, 1.0, -1, torch.zeros(10, 24))
    with pytest.raises(ValueError, match="res has shape"):
        scv.rms_norm_fwd(x, res=torch.zeros(4, 24))
    with pytest.raises(ValueError, match="w has type"):
        scv.rms_norm_fwd(x, torch.zeros(16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="rstd"):
        scv.rms_norm_bwd(x, x, torch.zeros(5))
    with pytest.raises(ValueError, match="takes h"):
        _lib.lat_rms_norm_bwd(x, None, x, q, s, torch.zeros(4), None, x)
    with pytest.raises(ValueError, match="values and its scales"):
        _lib.lat_rms_norm_fwd(x, None, None, 1e-6, y8=q)
    with pytest.raises(ValueError, match="q scale"):
        scv.q8_unpack(scv.Q8Rows(q, torch.zeros(4, 2, dtype=torch.uint8)))
    with pytest.raises(ValueError, match="q has type"):
        scv.q8_unpack(scv.Q8Rows(q.view(torch.uint8), s))
    with pytest.raises(ValueError, match="rows, not"):
        scv.embed_wgrad(ids, x, 10, out=torch.zeros(9, 16))
    km = scv.KernelMap.__new__(scv.KernelMap)
    km.c = _lib.lat_kmap()
    km.k3 = km.c.k3 = 27
    km.c.n_in, km.c.n_out = 4, 5
    with pytest.raises(ValueError, match="dy has shape"):
        scv.conv_wgrad_q8(scv.Q8Rows(q, s), x, km)
    with pytest.raises(ValueError, match="dw has shape"):
        _lib.lat_sconv_wgrad_q8(q, s, torch.zeros(5, 16), km.c, torch.zeros(27, 16, 8, dtype=f32))


def test_status_bit_of_a_bad_id(lib):
    assert scv.lat_status_string(1024) == "token id out of range"
    assert "LAT_ERR_BAD_ID" in str(scv.LatticeError(1024))


def _map(n_in=10, n_out=10, capacity=100):
    km = _lib.lat_kmap()
    km.k3, km.n_out, km.n_in, km.pair_capacity = 27, n_out, n_in, capacity
    km.nbr, km.perm, km.tile_mask, km.pair_off, km.pair_in, km.pair_out = (P(4096),) * 6
    return km


@pytest.mark.parametrize("cin,cout,dt", [(64, 64, 1), (128, 128, 2), (16, 16, 0), (40, 24, 2)])
def test_weight_gradient_from_8bit_rows_refuses_a_misaligned_workspace(lib, cin, cout, dt):
    """The partials are stored 32 bytes at a time, from the workspace's beginning."""
    km = _map()
    need = lib.lat_sconv_wgrad_q8_ws_bytes(cin, cout, ctypes.byref(km), dt)
    for off in (4, 8, 16, 24, 48):
        assert lib.lat_sconv_wgrad_q8(A, B, cin, C, cout, ctypes.byref(km), P(16384), dt, P((1 << 20) + off), need + 64,
                                      None, None) == WORKSPACE, off


@pytest.mark.parametrize("cin,cout,dt", [(64, 64, 1), (16, 16, 0)])
def test_weight_gradient_from_8bit_rows_refuses_null_gradient_rows(lib, cin, cout, dt):
    assert lib.lat_sconv_wgrad_q8(A, B, cin, None, cout, ctypes.byref(_map()), P(16384), dt, P(1 << 20), 1 << 30, None,
                                  None) == ARG
