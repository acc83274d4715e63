"""The 8-bit projection operators on the GPU against plain implementations (-m gpu): codes and scale
bytes bit for bit, products bit for bit where float holds every partial sum and within the error of
float accumulation elsewhere, and the whole run norm -> product -> compressor against the oracle on
the values the codes stand for."""

import numpy as np
import pytest
import torch

import quant_ref as ref
from compressed_kv_sparse_compressor_gb300 import abi, configs, fp8
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def guarded(n, k, rows=1):
    """(q, scale) buffers filled with 0xA5, and a check that what is no value stayed so."""
    qf = torch.full((n + 1, ref.up(k, 16)), 0xA5, dtype=torch.uint8, device="cuda")
    nb = -(-n // rows)
    sf = torch.full((nb + 1, fp8.scale_bytes(k)), 0xA5, dtype=torch.uint8, device="cuda")

    def check():
        assert (qf[n] == 0xA5).all() and (qf[:, k:] == 0xA5).all()
        assert (sf[nb] == 0xA5).all() and (sf[:, -(-k // 128):] == 0xA5).all()
    return qf[:n, :k].view(torch.float8_e4m3fn) if k % 16 == 0 else qf[:n, :k], sf[:nb], check


# ---- norm --------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d,residual,gain", [
    (1, 4096, True, True), (3, 1, False, True), (5, 7, True, False), (2, 127, True, True), (4, 128, False, False),
    (3, 129, True, True), (33, 1544, False, True), (17, 1541, True, True), (9, 4104, True, True),
    (300, 4096, True, True), (2, 8192, True, False), (2, 8200, True, True), (3, 16392, False, True),
    (2, 32768, True, True), (2, 32767, True, True),
])
def test_norm_matches_the_definition_bit_for_bit(dtype, n, d, residual, gain):
    g = gen(1000 + n + d)
    x = (randn(g, n, d) * torch.exp(randn(g, d))).to(dtype)
    r = (3 * randn(g, n, d)).to(dtype) if residual else None
    w = 1 + 0.1 * randn(g, d) if gain else None
    q, scale, check = guarded(n, d)
    h = torch.empty_like(x)
    y = torch.empty_like(x)
    fp8.rmsnorm(x, w, residual=r, residual_out=h, eps=EPS, q=q, scale=scale, y=y)
    wh, wy = ref.rmsnorm(x, r, w, EPS)
    wq, ws = ref.quantise(wy, 1)
    assert torch.equal(h, wh)
    assert torch.equal(y, wy.to(dtype))
    assert torch.equal(scale[:, :-(-d // 128)], ws)
    assert torch.equal(q.view(torch.uint8), wq)
    check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(512, 4096), (600, 4104), (513, 1024), (521, 256), (700, 100), (515, 8192), (512, 7168),
                                 (530, 1541), (512, 16392), (512, 5001), (900, 515), (600, 1285), (512, 16391)])
def test_norm_of_many_rows_bit_for_bit(dtype, n, d):
    # the forms for many rows: rows that fill their threads and rows that do not, several rows to a block
    g = gen(7 * n + d)
    x, r, w = randn(g, n, d).to(dtype), (3 * randn(g, n, d)).to(dtype), 1 + 0.1 * randn(g, d)
    q, scale, check = guarded(n, d)
    h = torch.empty_like(x)
    fp8.rmsnorm(x, w, residual=r, residual_out=h, eps=EPS, q=q, scale=scale)
    wh, wy = ref.rmsnorm(x, r, w, EPS)
    wq, ws = ref.quantise(wy, 1)
    assert torch.equal(h, wh)
    assert torch.equal(scale[:, :-(-d // 128)], ws)
    assert torch.equal(q.view(torch.uint8), wq)
    check()


def test_norm_strided_and_in_place():
    g = gen(3)
    n, d = 19, 520
    big = randn(g, n, 1200).bfloat16()
    x, r = big[:, 3:3 + d], big[:, 600:600 + d]                 # x starts 6 bytes off: the unaligned form
    wh, wy = ref.rmsnorm(x, r, None, EPS)
    wq, ws = ref.quantise(wy, 1)
    rest = big.clone()
    q, scale = fp8.rmsnorm(x, residual=r, residual_out=r, eps=EPS)
    assert torch.equal(r, wh) and torch.equal(q.view(torch.uint8), wq) and torch.equal(scale[:, :5], ws)
    rest[:, 600:600 + d] = wh
    assert torch.equal(big, rest)
    xx, rr = randn(g, 600, 1032), randn(g, 600, 1032)            # over x itself, and a residual added to itself
    wh, wy = ref.rmsnorm(xx, rr, None, EPS)
    q, scale = fp8.rmsnorm(xx, residual=rr, residual_out=xx, eps=EPS)
    assert torch.equal(xx, wh) and torch.equal(q.view(torch.uint8), ref.quantise(wy, 1)[0])
    wh, wy = ref.rmsnorm(xx, xx, None, EPS)
    q, scale = fp8.rmsnorm(xx, residual=xx, residual_out=xx, eps=EPS)
    assert torch.equal(xx, wh) and torch.equal(q.view(torch.uint8), ref.quantise(wy, 1)[0])
    # without the 8-bit output: the plain fused norm
    x = randn(g, n, d)
    y = torch.empty_like(x)
    a = abi.RmsnormArgs(n, d, abi.DS4C_F32, EPS, x.data_ptr(), None, None, y.data_ptr(), d, 0, 0, d)
    assert abi.ds4c_rmsnorm_quant(a, torch.cuda.current_stream().cuda_stream) == abi.DS4C_OK
    assert torch.equal(y, ref.rmsnorm(x, None, None, EPS)[1])
    # no rows
    q, scale = fp8.rmsnorm(x[:0])
    assert q.shape == (0, d) and scale.shape == (0, 8)


@pytest.mark.parametrize("d", [256, 1000, 4096])
def test_norm_of_extreme_rows(d):
    """Rows of zeros, of one value, of tiny and of huge values (squares beyond float), with an infinity,
    with NaN."""
    x = torch.zeros(8, d, device="cuda")
    x[1] = 1.0
    x[2, 5] = 1e-30
    x[3] = 1e30 * torch.linspace(-1, 1, d, device="cuda")
    x[4] = 3.0e38
    x[5] = 1.0
    x[5, 7] = float("inf")
    x[6] = 1.0
    x[6, 7] = float("nan")
    x[7] = torch.linspace(-1, 1, d, device="cuda") * 1e14
    q, scale = fp8.rmsnorm(x, eps=EPS)
    wq, ws = ref.quantise(ref.rmsnorm(x, None, None, EPS)[1], 1)
    nb = -(-d // 128)
    assert torch.equal(scale[:, :nb], ws)
    a, b = q.view(torch.uint8), wq
    nan = (b & 0x7F) == 0x7F
    assert torch.equal((a & 0x7F) == 0x7F, nan)
    assert torch.equal(a[~nan], b[~nan])
    assert nan[5].sum() == 1 and nan[6].all() and not nan[:5].any() and not nan[7].any()


# ---- weights -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(1, 1), (1, 4096), (127, 129), (128, 128), (129, 127), (300, 1541), (64, 1544),
                                 (1024, 4096)])
def test_weight_quantisation_bit_for_bit(dtype, n, k):
    g = gen(n * 7 + k)
    w = (0.02 * randn(g, n, k) * torch.exp(2 * randn(g, n, 1))).to(dtype)
    w[n // 2, k // 2] = float("nan") if n > 100 else 0.0
    q, scale, check = guarded(n, k, 128)
    fp8.quantize_weight(w, q, scale)
    wq, ws = ref.quantise(w.float(), 128)
    assert torch.equal(scale[:, :-(-k // 128)], ws)
    a, nan = q.view(torch.uint8), (wq & 0x7F) == 0x7F
    assert torch.equal((a & 0x7F) == 0x7F, nan) and torch.equal(a[~nan], wq[~nan])
    check()


def test_scale_rule_at_its_borders():
    """amax one float below, at and above 448 * 2^e for every e that bf16 / float hold."""
    e = torch.arange(-135, 119, device="cuda")
    top = (448 * ref.pow2(e)).float()
    w = torch.stack([torch.nextafter(top, torch.zeros_like(top)), top,
                     torch.nextafter(top, torch.full_like(top, float("inf")))], 1).reshape(-1, 1)
    w = torch.cat([w, torch.tensor([[1e-45], [3.4e38], [0.0]], device="cuda")])
    rows = w.repeat(1, 128).repeat_interleave(128, 0)
    got = fp8.quantize_weight(rows)
    wq, ws = ref.quantise(rows, 128)
    assert torch.equal(got.scale[:, :1], ws)
    assert torch.equal(got.q.view(torch.uint8), wq)


# ---- product -----------------------------------------------------------------------------------

def whole(g, n, k, rows, spread=2):
    """Codes of -2 .. 2 and scales 2^-spread .. 2^spread: products and sums that float holds exactly."""
    q, scale = fp8.empty(n, k, "cuda", rows)
    q.copy_(torch.randint(-2, 3, (n, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn))
    scale.copy_(torch.randint(127 - spread, 128 + spread, scale.shape, generator=g, device="cuda"))
    return q, scale


SHAPES = [
    (1, [1], 1), (1, [16], 16), (1, [1000], 4096), (2, [130], 144), (7, [129], 129), (15, [128], 512), (16, [256], 640),
    (17, [127], 1000), (31, [64, 3], 257), (32, [1024, 1024, 256, 256], 4096), (33, [500, 1], 1541), (64, [640], 2048),
    (65, [384, 128, 5], 1153), (127, [129], 520), (128, [256], 1024), (129, [1000], 1541), (200, [1024, 256], 520),
    (255, [300], 4096), (256, [128], 128), (257, [257], 2049), (437, [1000], 1541), (1000, [77, 130, 512, 1], 900),
    (2048, [1024, 1024, 256, 256], 4096), (5000, [520], 392), (5, [300], 20000), (100, [200, 40], 33000), (600, [2600], 9000),
    (64, [20000], 640), (129, [10000], 300), (3000, [4096], 130),
]


@pytest.mark.parametrize("m,ns,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product_of_whole_numbers_is_exact(m, ns, k, dtype):
    """Every code's place, every scale's place, every tail: sums below 2^24 steps of 2^-4 are exact in any order."""
    g = gen(m * 31 + k)
    q, scale = whole(g, m, k, 1)
    ws = [whole(g, n, k, 128) for n in ns]
    # outputs inside wider rows, a guard behind the last one
    full = [torch.full((m + 1, n + 5), 7.0, dtype=dtype, device="cuda") for n in ns]
    out = [f[:m, :n] for f, n in zip(full, ns)]
    fp8.Linear([fp8.Fp8Weight(*w) for w in ws])(q, scale, out)
    a = ref.values(q.view(torch.uint8), scale, 1)
    for (wq, wsc), o, f, n in zip(ws, out, full, ns):
        want = a @ ref.values(wq.view(torch.uint8), wsc, 128).T
        assert want.abs().max() < 2 ** 20 or m * n == 0
        assert torch.equal(o, want.float().to(dtype))
        assert (f[m] == 7).all() and (f[:, n:] == 7).all()


@pytest.mark.parametrize("m,ns,k,pad,off", [(700, [1000, 258], 8192, 6, 0), (701, [1000], 8192, 6, 2), (2050, [384], 640, 0, 0),
                                            (2050, [386, 385], 640, 4, 2), (999, [514], 512, 5, 1), (3001, [2], 256, 2, 0)])
def test_bfloat16_outputs_at_even_and_odd_places(m, ns, k, pad, off):
    """Outputs inside wider matrices at even and odd places and pitches: rounded once, nothing beside them."""
    g = gen(m + k + pad)
    q, scale = whole(g, m, k, 1)
    ws = [whole(g, n, k, 128) for n in ns]
    full = [torch.full((m + 1, n + pad + off), 7.0, dtype=torch.bfloat16, device="cuda") for n in ns]
    out = [f[:m, off:off + n] for f, n in zip(full, ns)]
    fp8.Linear([fp8.Fp8Weight(*w) for w in ws])(q, scale, out)
    a = ref.values(q.view(torch.uint8), scale, 1)
    for (wq, wsc), o, f, n in zip(ws, out, full, ns):
        assert torch.equal(o, (a @ ref.values(wq.view(torch.uint8), wsc, 128).T).float().bfloat16())
        assert (f[m] == 7).all() and (f[:, :off] == 7).all() and (f[:, off + n:] == 7).all()


@pytest.mark.parametrize("m,ns,k", [(1, [1024, 256], 4096), (3, [200], 8192), (33, [1024], 1541), (200, [640], 4096),
                                    (700, [1000], 8192), (2100, [384], 7168), (2, [256], 32768),
                                    (900, [2048], 12000)])
def test_product_error_is_that_of_float_sums(m, ns, k):
    """K products, each exact, added in float in an unknown order: every addition is off by at most 2^-23
    of a partial sum (2^-24 rounded to nearest), and a partial sum by at most the sum of magnitudes."""
    g = gen(m + k)
    q, scale = fp8.rmsnorm(randn(g, m, k) * torch.exp(randn(g, k)))
    ws = [fp8.quantize_weight(0.02 * randn(g, n, k)) for n in ns]
    outs = fp8.Linear(ws)(q, scale)
    a = ref.values(q.view(torch.uint8), scale, 1)
    for w, o in zip(ws, outs):
        wv = ref.values(w.q.view(torch.uint8), w.scale, 128)
        want, mag = a @ wv.T, a.abs() @ wv.abs().T
        assert ((o.double() - want).abs() <= k * 2.0 ** -23 * mag).all()
        # an accumulator takes at most 4096 values in steps of 32, 128 additions, and the partial sums of
        # independent products are in norm no larger than the whole: 128 * 2^-23, were all errors one way
        assert (o.double() - want).norm() <= 128 * 2.0 ** -23 * want.norm()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_product_with_extreme_scales_and_nan(m):
    g = gen(m)
    n, k = 260, 700
    q, scale = whole(g, m, k, 1)
    wq, wsc = whole(g, n, k, 128)
    scale[:, :] = 127 - 100
    wsc[:, :] = 127 + 99
    scale[m // 2, 1] = 0                               # 2^-127
    lin = fp8.Linear([fp8.Fp8Weight(wq, wsc)])
    got = lin(q, scale)[0]
    a, w = ref.values(q.view(torch.uint8), scale, 1), ref.values(wq.view(torch.uint8), wsc, 128)
    want = a @ w.T
    # float does not hold the block at 2^-127 next to the others: the bound of float sums for its row
    assert ((got.double() - want).abs() <= k * 2.0 ** -23 * (a.abs() @ w.abs().T)).all()
    rest = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(got[rest], want[rest].float())
    # a NaN code poisons its row or column, a scale byte of 255 the outputs of its block
    q.view(torch.uint8)[0, 5] = 0x7F
    wq.view(torch.uint8)[n - 1, k - 1] = 0xFF
    wsc[1, 2] = 255
    got = lin(q, scale)[0]
    want = ref.values(q.view(torch.uint8), scale, 1) @ ref.values(wq.view(torch.uint8), wsc, 128).T
    assert torch.equal(got.isnan(), want.isnan())
    assert got[0].isnan().all() and got[:, 128:256].isnan().all() and got[:, n - 1].isnan().all()
    # rows and columns behind the last have no part in it: pitches' padding and guards full of NaN
    fullq = torch.full((m + 3, ref.up(k, 16)), 0x7F, dtype=torch.uint8, device="cuda")
    fulls = torch.full((m + 3, fp8.scale_bytes(k)), 255, dtype=torch.uint8, device="cuda")
    q2, s2 = whole(g, m, k, 1)
    fullq[:m, :k] = q2.view(torch.uint8)
    fulls[:m, :6] = s2[:, :6]
    wq2, wsc2 = whole(g, n, k, 128)
    a = fp8.Linear([fp8.Fp8Weight(wq2, wsc2)])
    wide = a(fullq[:m, :k], fulls[:m])[0]
    assert torch.equal(wide, a(q2, s2)[0]) and not wide.isnan().any()


@pytest.mark.parametrize("m", [1, 40, 600])
@pytest.mark.parametrize("a,w", [(0, 254), (254, 0), (1, 253), (127, 127)])
def test_product_at_the_ends_of_the_scales(m, a, w):
    """Scales 2^-127 and 2^127 that cancel: whole numbers again."""
    g = gen(m + a)
    n, k = 300, 660
    q, scale = whole(g, m, k, 1)
    wq, wsc = whole(g, n, k, 128)
    scale.fill_(a)
    wsc.fill_(w)
    want = q.double() @ wq.double().T
    assert torch.equal(fp8.Linear([fp8.Fp8Weight(wq, wsc)])(q, scale)[0], want.float())


def test_no_rows():
    w = fp8.quantize_weight(torch.ones(4, 32, device="cuda"))
    q, scale = fp8.empty(0, 32)
    assert fp8.Linear([w])(q, scale)[0].shape == (0, 4)


def test_same_result_every_time_on_two_streams_and_in_a_graph():
    g = gen(9)
    m, k = 32, 4096
    x, res = randn(g, m, k).bfloat16(), randn(g, m, k).bfloat16()
    gain = 1 + 0.1 * randn(g, k)
    ws = [fp8.quantize_weight(0.02 * randn(g, n, k)) for n in (1024, 256)]
    lin = fp8.Linear(ws)
    q0, s0 = fp8.rmsnorm(x, gain, residual=res)
    want = [o.clone() for o in lin(q0, s0)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):                                     # two runs at once, nothing shared but the inputs
        for st in streams:
            with torch.cuda.stream(st):
                q, s = fp8.rmsnorm(x, gain, residual=res)
                outs.append(lin(q, s))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    # captured, then replayed on other data
    q, s = fp8.empty(m, k)
    o = [torch.empty(m, w.shape[0], device="cuda") for w in ws]
    xs = x.clone()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        fp8.rmsnorm(xs, gain, residual=res, q=q, scale=s)
        lin(q, s, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        fp8.rmsnorm(xs, gain, residual=res, q=q, scale=s)
        lin(q, s, o)
    for seed in (1, 2):
        xs.copy_(randn(gen(seed), m, k))
        graph.replay()
        q1, s1 = fp8.rmsnorm(xs, gain, residual=res)
        assert all(torch.equal(a, b) for a, b in zip(o, lin(q1, s1)))
    xs.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_two_threads_on_two_streams():
    """The handle of the weights is shared, each thread has its own rows, outputs and stream."""
    import threading
    g = gen(33)
    k = 1544
    lin = fp8.Linear([fp8.quantize_weight(0.02 * randn(g, n, k)) for n in (520, 64)])
    xs = [[randn(g, m, k) for m in (1, 50, 300)] for _ in range(2)]
    want = [[lin(*fp8.rmsnorm(x)) for x in rows] for rows in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(60):
                for x, w in zip(xs[i], want[i]):
                    got = lin(*fp8.rmsnorm(x))
                    st.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, w)):
                        wrong.append((i, x.shape))
            st.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_back_to_back_calls_read_what_the_one_before_wrote():
    """Weights requantised, rows renormalised and multiplied, again and again into the same buffers with nothing
    in between: each product equals the one of its own inputs with a wait after every call."""
    g = gen(21)
    m, n, k = 48, 640, 1032
    xs, ws = [randn(g, m, k).bfloat16() for _ in range(6)], [0.02 * randn(g, n, k) for _ in range(6)]
    want = []
    for x, w in zip(xs, ws):
        wq = fp8.quantize_weight(w)
        torch.cuda.synchronize()
        q, s = fp8.rmsnorm(x)
        torch.cuda.synchronize()
        want.append(fp8.Linear([wq])(q, s)[0])
        torch.cuda.synchronize()
    q, s = fp8.empty(m, k)
    wq = fp8.Fp8Weight(*fp8.empty(n, k, "cuda", 128))
    lin = fp8.Linear([wq])
    outs = []
    for _ in range(20):
        for x, w in zip(xs, ws):
            fp8.quantize_weight(w, wq.q, wq.scale)
            fp8.rmsnorm(x, q=q, scale=s)
            outs.append(lin(q, s)[0])
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 6]), i


# ---- the layer ---------------------------------------------------------------------------------

def _layers(ratio, T, n_seq=1, **kw):
    """A float32 layer whose weights are the values of the quantised ones, and the quantised layer."""
    from compressed_kv_sparse_compressor_gb300.layer import DeviceLayer
    shape = configs.LayerShape(**{**dict(d_model=520, head_dim=128, n_rot=64, idx_head_dim=64, n_heads=8, ratio=ratio,
                                         top_k=8, dtype="f32", w_std=0.04), **kw})
    made = []
    for _ in range(2):
        dl = DeviceLayer(shape, comp_cap=T, idx_cap=T, n_seq=n_seq, max_rows=max(T, n_seq), with_prequant=True)
        dl.state_init()
        made.append(dl)
    lanes = [configs.lane_weights(shape, 5, 0, lane, device="cuda", gamma_std=0.1)
             for lane in (("attn", "idx") if ratio == 4 else ("attn",))]
    quant = [[fp8.quantize_weight(t) for t in w[:2]] for w in lanes]
    made[0].set_weights(*[[ref.values(t.q.view(torch.uint8), t.scale, 128).float() for t in tq] + list(w[2:])
                          for tq, w in zip(quant, lanes)])
    made[1].set_weights_quant(*[list(tq) + list(w[2:]) for tq, w in zip(quant, lanes)])
    return shape, made[0], made[1]


def _close(a, b):
    """Two layers' states after the same tokens, with the path's tolerance for float-accumulated values."""
    for name in ("attn_kv", "attn_score", "attn_pre", "idx_kv", "idx_score", "idx_comp"):
        u, v = getattr(a, name), getattr(b, name)
        if u is None:
            continue
        fin = torch.isfinite(u)
        assert torch.equal(fin, torch.isfinite(v)), name
        assert ((u - v)[fin].abs() <= 1e-4 + 2e-3 * u[fin].abs()).all(), name


@pytest.mark.parametrize("ratio,T,kw", [(4, 300, {}), (128, 300, {}), (4, 37, dict(d_model=1544)),
                                        (4, 1100, dict(d_model=512, head_dim=512, idx_head_dim=128, n_heads=64, dtype="bf16"))])
def test_layer_prefill_from_the_norm_to_the_compressed_rows(ratio, T, kw):
    """norm -> 8-bit rows -> four products -> compressor, in two ragged chunks, against the float layer on
    the values the codes stand for."""
    shape, plain, quant = _layers(ratio, T, **{**kw, "dtype": "f32"})
    g = gen(T)
    x, res = randn(g, T, shape.d_model).bfloat16(), randn(g, T, shape.d_model).bfloat16()
    gain = 1 + 0.1 * randn(g, shape.d_model)
    pos = 0
    for n in (T // 3 + 1, T - T // 3 - 1):
        q, scale = fp8.rmsnorm(x[pos:pos + n], gain, residual=res[pos:pos + n])
        quant.compress_prefill_quant(q, scale, pos)
        plain.compress_prefill(ref.values(q.view(torch.uint8), scale, 1).float().contiguous(), pos)
        pos += n
    quant.sync()
    _close(plain, quant)


def test_layer_decode_steps():
    shape, plain, quant = _layers(4, 64, n_seq=9)
    g = gen(77)
    pos = [3 * b for b in range(9)]
    for b in range(9):                                      # staggered prefixes through both layers
        if pos[b]:
            q, scale = fp8.rmsnorm(randn(g, pos[b], shape.d_model))
            v = ref.values(q.view(torch.uint8), scale, 1).float().contiguous()
            for dl, call in ((plain, None), (quant, None)):
                view = dl.seq_view(b)
                s = torch.cuda.current_stream().cuda_stream
                if dl is plain:
                    st = abi.ds4c_compress_prefill(dl.cfg, dl.attn_w, dl.idx_w, view, v.data_ptr(), pos[b], 0,
                                                   dl.ws.data_ptr(), dl.ws_bytes, s)
                else:
                    st = abi.ds4c_compress_prefill_quant(dl.cfg, dl.attn_wq, dl.idx_wq, view, q.data_ptr(),
                                                         scale.data_ptr(), pos[b], 0, dl.ws.data_ptr(), dl.ws_bytes, s)
                assert st == abi.DS4C_OK
    for step in range(6):
        q, scale = fp8.rmsnorm(randn(g, 9, shape.d_model))
        quant.compress_decode_quant(q, scale, [p + step for p in pos])
        plain.compress_decode(ref.values(q.view(torch.uint8), scale, 1).float().contiguous(), [p + step for p in pos])
    quant.sync()
    _close(plain, quant)


def test_layer_refusals():
    shape, _, quant = _layers(4, 16)
    wa, wi = (configs.lane_weights(shape, 5, 0, lane, device="cuda") for lane in ("attn", "idx"))
    q, scale = fp8.empty(4, shape.d_model)
    for bad in (lambda: quant.set_weights_quant((wa[0][:-1],) + wa[1:], wi), lambda: quant.set_weights_quant(wi, wi),
                lambda: quant.set_weights_quant(wa[:2] + (wa[2][:3], wa[3]), wi),
                lambda: quant.set_weights_quant(wa[:3] + (wa[3][:-4],), wi),
                lambda: quant.compress_prefill_quant(*fp8.empty(4, shape.d_model + 16), 0),
                lambda: quant.compress_decode_quant(q, scale, [0, 1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(abi.Ds4cError):
        quant.compress_prefill_quant(*fp8.empty(68, shape.d_model), 0)      # past the state's capacity


def test_layer_refuses_a_bias_or_gain_of_another_type():
    # the library reads both as floats: of a narrower type it would read past their end
    shape, _, quant = _layers(4, 16)
    wa, wi = (configs.lane_weights(shape, 5, 0, lane, device="cuda") for lane in ("attn", "idx"))
    for dt in (torch.bfloat16, torch.float16, torch.float64):
        for bad in (wa[:2] + (wa[2].to(dt), wa[3]), wa[:3] + (torch.ones(shape.head_dim, dtype=dt, device="cuda"),)):
            with pytest.raises(ValueError):
                quant.set_weights_quant(bad, wi)


# ---- refusals of the torch calls -----------------------------------------------------------------

def test_refusals_of_the_torch_calls():
    x = torch.zeros(4, 256, device="cuda")
    q, scale = fp8.empty(4, 256)
    for bad in (lambda: fp8.rmsnorm(x.half()), lambda: fp8.rmsnorm(x[0]), lambda: fp8.rmsnorm(x.cpu()),
                lambda: fp8.rmsnorm(x.T), lambda: fp8.rmsnorm(x, residual=x.bfloat16()),
                lambda: fp8.rmsnorm(x, residual=x[:3]), lambda: fp8.rmsnorm(x, torch.ones(255, device="cuda")),
                lambda: fp8.rmsnorm(x, torch.ones(256)), lambda: fp8.rmsnorm(x, q=q),
                lambda: fp8.rmsnorm(x, q=q[:3], scale=scale[:3]), lambda: fp8.rmsnorm(x, q=q, scale=scale[:, :2]),
                lambda: fp8.quantize_weight(x.half()), lambda: fp8.quantize_weight(x, q, scale),
                lambda: fp8.Fp8Weight(q, scale), lambda: fp8.Linear([])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(abi.Ds4cError):
        fp8.rmsnorm(x, eps=0.0)
    with pytest.raises(abi.Ds4cError):
        fp8.rmsnorm(x[:1].expand(4, 256))                   # rows that overlap
    with pytest.raises(abi.Ds4cError):
        fp8.rmsnorm(torch.zeros(4, 258, device="cuda"), q=torch.zeros(4, 272, dtype=torch.uint8, device="cuda")[:, 1:259],
                    scale=torch.zeros(4, 4, dtype=torch.uint8, device="cuda"))   # rows off their 16 bytes
    w = fp8.quantize_weight(x)
    lin = fp8.Linear([w])
    for bad in (lambda: lin(q[:, :128], scale), lambda: lin(q, scale, [torch.zeros(4, 5, device="cuda")]),
                lambda: lin(q, scale, [torch.zeros(4, 4)]), lambda: lin(q, scale, []),
                lambda: lin(q, scale, dtype=torch.float16),
                lambda: fp8.Linear([w, fp8.quantize_weight(x[:, :128])])):
        with pytest.raises(ValueError):
            bad()


def test_layer_keeps_its_weights_when_new_ones_are_refused():
    """A call that raises on the second lane leaves both lanes as they were, not one of each."""
    shape, _, quant = _layers(4, 16)
    wa, wi = (configs.lane_weights(shape, 6, 0, lane, device="cuda") for lane in ("attn", "idx"))
    before = bytes(quant.attn_wq), bytes(quant.idx_wq)
    for bad in (None, wa, (wi[0][:-1],) + wi[1:], wi[:2] + (wi[2].double(), wi[3])):
        with pytest.raises((ValueError, TypeError)):
            quant.set_weights_quant(wa, bad)
        assert (bytes(quant.attn_wq), bytes(quant.idx_wq)) == before
    quant.set_weights_quant(wa, wi)
    after = bytes(quant.attn_wq), bytes(quant.idx_wq)
    assert after[0] != before[0] and after[1] != before[1]


@pytest.mark.parametrize("n,d", [(400, 256), (300, 4096), (300, 1001), (600, 2056)])
def test_norm_whose_reciprocal_root_is_subnormal(n, d):
    """Rows with a root mean square from 2^125 to 2^128: rstd is a subnormal float near 2^-127, rounded once."""
    g = gen(n + d)
    x = torch.rand(n, d, generator=g, device="cuda") + 0.5
    x *= torch.where(torch.rand(n, d, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = (x * (torch.exp2(125.0 + 2.4 * torch.rand(n, 1, generator=g, device="cuda", dtype=torch.float64)))).float()
    assert torch.isfinite(x).all()
    q, scale, check = guarded(n, d)
    y = torch.empty_like(x)
    fp8.rmsnorm(x, eps=EPS, q=q, scale=scale, y=y)
    wy = ref.rmsnorm(x, None, None, EPS)[1]
    wq, ws = ref.quantise(wy, 1)
    assert torch.equal(y, wy)
    assert torch.equal(scale[:, :-(-d // 128)], ws)
    assert torch.equal(q.view(torch.uint8), wq)
    check()
