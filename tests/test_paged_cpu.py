"""Host validation of the attention over a paged cache: bad arguments refused before any launch."""

import pytest
import torch

from compressed_kv_sparse_compressor_gb300 import abi, paged
from compressed_kv_sparse_compressor_gb300 import build as build_mod

FAKE = 1 << 20          # an aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    abi.lib()


def pool(**kw):
    f = dict(rows=FAKE, pages=FAKE, pages_ld=8, n_pages=20, page_rows=64, max_pages=8)
    f.update(kw)
    return abi.PagePool(**f)


def call(raw=None, comp=None, ws=FAKE, ws_bytes=None, **kw):
    f = dict(n_seq=3, n_tok=10, n_heads=64, head_dim=512, window=0, ratio=0, scale=0.1, q=FAKE, out=2 * FAKE, q_token=64 * 512, q_head=512,
             out_token=64 * 512, out_head=512, start=FAKE, length=FAKE)
    f.update(kw)
    if ws_bytes is None:
        ws_bytes = abi.ds4c_paged_attn_workspace_bytes(3, 10, 64, 512)
    return abi.ds4c_paged_attn(abi.PagedAttnArgs(**f, raw=pool(**(raw or {})), comp=abi.PagePool() if comp is None else pool(**comp)),
                               ws, ws_bytes, None)


def test_refusals():
    nan = float("nan")
    assert abi.lib().ds4c_paged_attn(None, FAKE, 1 << 30, None) == abi.DS4C_ERR_NULL
    assert call(n_tok=0) == call(n_seq=0) == call(n_tok=0, q=None, out=None, ws=None) == abi.DS4C_OK
    for kw in (dict(q=None), dict(out=None), dict(start=None), dict(length=None), dict(raw=dict(rows=None)), dict(raw=dict(pages=None)),
               dict(ratio=4, comp=dict(rows=None)), dict(ratio=4, comp=dict(pages=None))):
        assert call(**kw) == abi.DS4C_ERR_NULL, kw
    for kw in (dict(n_seq=4097), dict(n_tok=(1 << 20) + 1), dict(n_heads=0), dict(n_heads=129), dict(head_dim=96), dict(head_dim=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=1e5), dict(window=1 << 31), dict(ratio=1 << 31),
               dict(q=FAKE + 8), dict(out=FAKE + 8), dict(start=FAKE + 2), dict(length=FAKE + 2), dict(q_token=64 * 512 + 4),
               dict(q_head=516), dict(out_token=64 * 512 + 4), dict(out_head=516), dict(out_head=504), dict(out_token=63 * 512),
               dict(ratio=4), dict(q_token=1 << 41), dict(q_token=0), dict(q_head=0), dict(out=FAKE)):
        assert call(**kw) == abi.DS4C_ERR_SHAPE, kw
    for kw in (dict(page_rows=8), dict(page_rows=48), dict(page_rows=2048), dict(page_rows=0), dict(n_pages=0), dict(n_pages=1 << 25),
               dict(pages_ld=7), dict(rows=FAKE + 8), dict(pages=FAKE + 2), dict(max_pages=(1 << 27) + 1, pages_ld=1 << 28)):
        assert call(raw=kw) == abi.DS4C_ERR_SHAPE, kw
        assert call(ratio=4, comp=kw) == abi.DS4C_ERR_SHAPE, kw
    need = abi.ds4c_paged_attn_workspace_bytes(3, 10, 64, 512)
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(ws_bytes=need - 1)):
        assert call(**kw) == abi.DS4C_ERR_WORKSPACE, kw
    for bad in ((4097, 1, 64, 512), (1, (1 << 20) + 1, 64, 512), (1, 1, 0, 512), (1, 1, 129, 512), (1, 1, 64, 500)):
        assert abi.ds4c_paged_attn_workspace_bytes(*bad) == 0
    assert abi.ds4c_paged_attn_workspace_bytes(0, 0, 1, 64) > 0


def test_python_refusals():
    q, cache = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        paged.attention(q, cache, i[None], i, i[:1])
    with pytest.raises(ValueError, match="bfloat16"):
        paged.attention(q.float(), cache, i[None], i, i[:1])


def test_packed_arguments_are_the_struct():
    a = abi.PagedAttnArgs.from_buffer_copy(paged._pack(*range(1, 7), 0.5, *range(8, 28)))
    assert [getattr(a, f) for f, _ in abi.PagedAttnArgs._fields_[:-2]] == [*range(1, 7), 0.5, *range(8, 16)]
    assert [getattr(p, f) for p in (a.raw, a.comp) for f, _ in abi.PagePool._fields_] == list(range(16, 28))
