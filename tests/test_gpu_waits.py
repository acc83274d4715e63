"""The kernels' bounded waits, in forms that fault and hang nothing (-m gpu): a wait that runs out gives the whole
warp one answer, raises the device error word and leaves the context usable."""

import pytest
import torch

import quant_ref as ref
from compressed_kv_sparse_compressor_gb300 import abi, configs, fp8
from gpu_util import device_layer, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    abi.check(abi.ds4c_test_set_wait_limit(0), "ds4c_test_set_wait_limit")


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("kernels", [abi.DS4C_WAITS_QUANT_MATMUL, abi.DS4C_WAITS_GEMM, abi.DS4C_WAITS_ATTENTION])
def test_lanes_that_see_different_things_get_one_answer(kernels):
    """Half of the lanes see what they wait for, the others never do: no lane may go on alone.  Then a barrier that
    nothing arrives on, and a complete one."""
    answers = torch.full((96,), -7, dtype=torch.int32, device="cuda")
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    assert abi.ds4c_test_set_wait_limit(20000) == abi.DS4C_OK                  # 20 us
    try:
        assert abi.ds4c_test_warp_wait(kernels, answers.data_ptr(), stream()) == abi.DS4C_OK
        assert abi.ds4c_sync_status(stream()) == abi.DS4C_ERR_DEVICE
    finally:
        assert abi.ds4c_test_set_wait_limit(0) == abi.DS4C_OK
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    assert answers.tolist() == [0] * 64 + [1] * 32


@pytest.mark.parametrize("m,n,k", [(1, 2560, 4096), (40, 512, 20000), (200, 1024, 4096), (300, 4096, 4096),
                                   (1500, 4096, 2176), (4096, 2560, 4096)])
def test_product_whose_waits_give_up(m, n, k):
    """The product in each of its forms with a limit of a few nanoseconds: its waits give up or not, as the copies
    come.  Either way it ends with nothing in flight, and with the default limit the same call is right."""
    g = torch.Generator(device="cuda").manual_seed(m + k)
    q, scale = fp8.empty(m, k)
    w = fp8.Fp8Weight(*fp8.empty(n, k, "cuda", 128))
    for codes, scales in ((q, scale), (w.q, w.scale)):
        codes.copy_(torch.randint(-2, 3, codes.shape, generator=g, device="cuda").float().to(torch.float8_e4m3fn))
        scales.copy_(torch.randint(126, 129, scales.shape, generator=g, device="cuda"))
    lin = fp8.Linear([w])
    want = (ref.values(q.view(torch.uint8), scale, 1) @ ref.values(w.q.view(torch.uint8), w.scale, 128).T).float()
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    out = [torch.empty(m, n, device="cuda")]
    assert abi.ds4c_test_set_wait_limit(1) == abi.DS4C_OK
    try:
        for _ in range(3):
            lin(q, scale, out)
            assert abi.ds4c_sync_status(stream()) in (abi.DS4C_OK, abi.DS4C_ERR_DEVICE)
    finally:
        assert abi.ds4c_test_set_wait_limit(0) == abi.DS4C_OK
    out[0].fill_(float("nan"))
    lin(q, scale, out)
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    assert torch.equal(out[0], want)


def test_products_right_behind_one_another():
    """Pairs of CTAs and single ones take turns on the same SMs with nothing in between: what one leaves behind in
    shared memory (an arrival of its last commits) would meet the barriers of the next."""
    g = torch.Generator(device="cuda").manual_seed(5)
    k = 640
    w = fp8.Linear([fp8.quantize_weight(torch.randint(-2, 3, (1024, k), generator=g, device="cuda").float())])
    rows = [fp8.rmsnorm(torch.randn(m, k, generator=g, device="cuda")) for m in (2000, 40, 1999, 1)]
    want = []
    for q, scale in rows:
        want.append(w(q, scale)[0])
        torch.cuda.synchronize()
    outs = [[w(q, scale)[0] for q, scale in rows] for _ in range(100)]
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 32, 300, 4096])
def test_projection_whose_waits_give_up(T):
    """The bf16 projection under the same limit, prefill chunks and decode-sized ones."""
    shape = configs.LayerShape(d_model=4096, head_dim=512, n_rot=64, idx_head_dim=128, n_heads=64, ratio=4, top_k=16,
                               dtype="bf16")
    dl, _, _ = device_layer(shape, comp_cap=T // 4 + 1, idx_cap=T // 4 + 1, max_rows=T, seed=3)
    h = configs.hidden(shape, 3, T).cuda()
    rows = dl.ws[: T * 2560 * 4].view(torch.float32)                    # what the projection wrote
    dl.compress_prefill(h, 0)
    dl.sync()
    want = rows.clone()
    assert abi.ds4c_test_set_wait_limit(1) == abi.DS4C_OK
    try:
        for _ in range(3):
            dl.compress_prefill(h, 0)
            assert abi.ds4c_sync_status(stream()) in (abi.DS4C_OK, abi.DS4C_ERR_DEVICE)
    finally:
        assert abi.ds4c_test_set_wait_limit(0) == abi.DS4C_OK
    rows.fill_(float("nan"))
    dl.compress_prefill(h, 0)
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    assert torch.equal(rows, want)


@pytest.mark.parametrize("n_seq,T,D", [(1, 700, 512), (1, 200, 128), (5, 1, 512)])
def test_attention_whose_waits_give_up(n_seq, T, D):
    """The tensor-core attention under the same limit: prefill queries of two head widths, a decode step."""
    shape = configs.LayerShape(d_model=256, head_dim=D, n_rot=64, idx_head_dim=64, n_heads=64, ratio=4, top_k=300,
                               dtype="bf16")
    cap = 500
    dl, _, _ = device_layer(shape, comp_cap=cap, idx_cap=cap, n_seq=n_seq, max_rows=max(T, n_seq), seed=5)
    assert abi.ds4c_attn_uses_tensor_cores(dl.cfg) == 1
    g = torch.Generator(device="cuda").manual_seed(D)
    dl.raw.copy_(torch.randn(dl.raw.shape, generator=g, device="cuda"))
    dl.attn_split.view(torch.bfloat16).copy_(torch.randn(dl.attn_split.shape, generator=g, device="cuda"))
    n = n_seq * T
    pos = [1200] if n_seq == 1 else [1200 + 50 * b for b in range(n_seq)]
    q = torch.randn(n, 64, D, generator=g, device="cuda")
    new = torch.randn(n, D, generator=g, device="cuda")
    topk = torch.arange(300, dtype=torch.int32, device="cuda").repeat(n, 1)
    want, out = torch.empty_like(q), torch.empty_like(q)
    dl.attention(q, new, topk, pos, n_seq, T, want, commit_ring=False)
    dl.sync()
    assert torch.isfinite(want).all()
    assert abi.ds4c_test_set_wait_limit(1) == abi.DS4C_OK
    try:
        for _ in range(2):
            dl.attention(q, new, topk, pos, n_seq, T, out, commit_ring=False)
            assert abi.ds4c_sync_status(stream()) in (abi.DS4C_OK, abi.DS4C_ERR_DEVICE)
    finally:
        assert abi.ds4c_test_set_wait_limit(0) == abi.DS4C_OK
    out.fill_(float("nan"))
    dl.attention(q, new, topk, pos, n_seq, T, out, commit_ring=False)
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    assert torch.equal(out, want)


def test_torch_calls_report_a_product_that_gave_up():
    answers = torch.empty(96, dtype=torch.int32, device="cuda")
    fp8.sync()
    assert abi.ds4c_test_set_wait_limit(20000) == abi.DS4C_OK
    try:
        assert abi.ds4c_test_warp_wait(abi.DS4C_WAITS_QUANT_MATMUL, answers.data_ptr(), stream()) == abi.DS4C_OK
        with pytest.raises(abi.Ds4cError) as e:
            fp8.sync("cuda")
        assert e.value.status == abi.DS4C_ERR_DEVICE
    finally:
        assert abi.ds4c_test_set_wait_limit(0) == abi.DS4C_OK
    fp8.sync(torch.device("cuda", 0))
    w = fp8.quantize_weight(torch.ones(8, 256, device="cuda"))
    q, scale = fp8.rmsnorm(torch.ones(3, 256, device="cuda"))
    out = fp8.Linear([w])(q, scale)[0]
    fp8.sync()
    assert torch.equal(out, torch.full_like(out, 256.0))
