"""Host validation of the 8-bit projection calls: sizes, and bad arguments refused before any launch."""

import pytest

from compressed_kv_sparse_compressor_gb300 import abi, configs, fp8
from compressed_kv_sparse_compressor_gb300 import build as build_mod

FAKE = 1 << 20          # an aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    abi.lib()


def test_pitches():
    for k, row, scale in ((1, 16, 4), (16, 16, 4), (17, 32, 4), (512, 512, 4), (513, 528, 8), (1541, 1552, 16),
                          (4096, 4096, 32), (1 << 18, 1 << 18, 2048)):
        assert abi.ds4c_quant_row_bytes(k) == fp8.row_bytes(k) == row
        assert abi.ds4c_quant_scale_bytes(k) == fp8.scale_bytes(k) == scale


def norm(**kw):
    a = abi.RmsnormArgs(4, 256, abi.DS4C_BF16, 1e-6, FAKE, None, None, None, 256, 0, 0, 0, None, FAKE, FAKE)
    for name, v in kw.items():
        setattr(a, name, v)
    return abi.ds4c_rmsnorm_quant(a, None)


def test_norm_refusals():
    assert norm(n=0) == abi.DS4C_OK                           # nothing to do
    for kw in (dict(x=None), dict(q=None), dict(scale=None), dict(q=None, scale=None)):
        assert norm(**kw) == abi.DS4C_ERR_NULL, kw
    for kw in (dict(d=0), dict(d=32769), dict(dtype=2), dict(eps=0.0), dict(eps=1e-13), dict(eps=float("nan")),
               dict(eps=2.0), dict(x=FAKE + 1), dict(x_ld=255), dict(residual=FAKE, residual_ld=255),
               dict(residual=FAKE + 1, residual_ld=256), dict(residual_out=FAKE + 64, residual_out_ld=255),
               dict(y_out=FAKE, y_ld=0), dict(gain=FAKE + 2), dict(q=FAKE + 8), dict(scale=FAKE + 2),
               dict(n=(1 << 24) + 1), dict(residual_out=FAKE, residual_out_ld=512),
               dict(residual=FAKE + 64, residual_ld=256, residual_out=FAKE + 64, residual_out_ld=264)):
        assert norm(**kw) == abi.DS4C_ERR_SHAPE, kw
    assert abi.lib().ds4c_rmsnorm_quant(None, None) == abi.DS4C_ERR_NULL


def test_weight_refusals():
    def call(n=4, k=256, dtype=abi.DS4C_F32, w=FAKE, ld=256, q=FAKE, scale=FAKE):
        return abi.ds4c_quant_weight(n, k, dtype, w, ld, q, scale, None)
    for kw in (dict(w=None), dict(q=None), dict(scale=None)):
        assert call(**kw) == abi.DS4C_ERR_NULL, kw
    for kw in (dict(n=0), dict(k=0), dict(n=(1 << 18) + 1), dict(k=(1 << 18) + 1, ld=1 << 19), dict(dtype=7), dict(ld=255),
               dict(w=FAKE + 2), dict(q=FAKE + 8), dict(scale=FAKE + 1)):
        assert call(**kw) == abi.DS4C_ERR_SHAPE, kw


def test_product_refusals():
    def call(m=4, k=256, a=FAKE, sa=FAKE, n_w=1, dtype=abi.DS4C_F32, **kw):
        f = dict(q=FAKE, scale=FAKE, out=FAKE, out_ld=64, n=64)
        f.update(kw)
        mats = (abi.QuantMatrix * 4)(*[abi.QuantMatrix(f["q"], f["scale"], f["out"], f["out_ld"], f["n"])] * 4)
        return abi.ds4c_quant_matmul(m, k, a, sa, mats, n_w, dtype, None)
    assert call(m=0) == abi.DS4C_OK
    assert call(m=0, a=None, out=None) == abi.DS4C_OK
    assert abi.ds4c_quant_matmul(4, 256, FAKE, FAKE, None, 1, abi.DS4C_F32, None) == abi.DS4C_ERR_NULL
    for kw in (dict(a=None), dict(sa=None), dict(q=None), dict(scale=None), dict(out=None)):
        assert call(**kw) == abi.DS4C_ERR_NULL, kw
    for kw in (dict(n_w=0), dict(n_w=5)):
        assert call(**kw) == abi.DS4C_ERR_UNSUPPORTED, kw
    for kw in (dict(m=(1 << 24) + 1), dict(k=0), dict(k=(1 << 18) + 1), dict(dtype=2), dict(n=0), dict(n=(1 << 18) + 1),
               dict(out_ld=63), dict(out=FAKE + 2), dict(q=FAKE + 8), dict(scale=FAKE + 2), dict(a=FAKE + 8),
               dict(sa=FAKE + 1)):
        assert call(**kw) == abi.DS4C_ERR_SHAPE, kw


def test_compress_refusals():
    shape = configs.C1.layer
    cfg = abi.LayerCfg(d_model=shape.d_model, head_dim=shape.head_dim, n_rot=shape.n_rot, idx_head_dim=shape.idx_head_dim,
                       n_heads=shape.n_heads, ratio=4, swa=shape.swa, top_k=shape.top_k, comp_cap=16, idx_cap=16,
                       dtype=abi.DS4C_F32, rms_eps=shape.rms_eps, attn_scale=shape.attn_scale,
                       rope_base=shape.rope_base)
    lane = abi.LaneState(FAKE, FAKE, FAKE, None, FAKE)
    st = abi.LayerState(FAKE, lane, lane)
    need = abi.ds4c_workspace_bytes(cfg, 64, 4)

    def weights(**kw):
        f = dict(wkv=FAKE, wkv_scale=FAKE, wgate=FAKE, wgate_scale=FAKE, ape=FAKE, norm=None)
        f.update(kw)
        return abi.LaneWeightsQuant(**f)
    w = weights()

    def prefill(aw=w, iw=w, h=FAKE, hs=FAKE, n=64, ws=FAKE, bytes=need):
        return abi.ds4c_compress_prefill_quant(cfg, aw, iw, st, h, hs, n, 0, ws, bytes, None)

    def decode(aw=w, iw=w, h=FAKE, hs=FAKE, n=4, ws=FAKE, bytes=need):
        return abi.ds4c_compress_decode_step_quant(cfg, aw, iw, st, h, hs, abi.u64_array([0] * n), n, ws, bytes, None)
    assert prefill(n=0) == abi.DS4C_OK
    assert prefill(n=68) == abi.DS4C_ERR_CAPACITY
    assert decode(n=1025) == abi.DS4C_ERR_UNSUPPORTED
    assert prefill(bytes=16) == decode(bytes=16) == abi.DS4C_ERR_WORKSPACE
    for call in (prefill, decode):
        assert call(ws=None) == abi.DS4C_ERR_WORKSPACE
        for kw in (dict(h=None), dict(hs=None), dict(aw=None), dict(iw=None)):
            assert call(**kw) == abi.DS4C_ERR_NULL, kw
        for kw in (dict(h=FAKE + 8), dict(hs=FAKE + 2)):
            assert call(**kw) == abi.DS4C_ERR_SHAPE, kw
        for name in ("wkv", "wkv_scale", "wgate", "wgate_scale", "ape"):
            assert call(aw=weights(**{name: None})) == abi.DS4C_ERR_NULL, name
            assert call(iw=weights(**{name: FAKE + 2})) == abi.DS4C_ERR_SHAPE, name


def test_warp_wait_refusals():
    assert abi.ds4c_test_warp_wait(abi.DS4C_WAITS_QUANT_MATMUL, None, None) == abi.DS4C_ERR_NULL
    assert abi.ds4c_test_warp_wait(abi.DS4C_WAITS_QUANT_MATMUL, FAKE + 2, None) == abi.DS4C_ERR_SHAPE
    assert abi.ds4c_test_warp_wait(99, FAKE, None) == abi.DS4C_ERR_UNSUPPORTED
