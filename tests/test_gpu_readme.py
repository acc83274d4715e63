"""The README's example of a layer over 8-bit projections, run as it stands (-m gpu)."""

import os
import re

import pytest
import torch

import quant_ref as ref
from compressed_kv_sparse_compressor_gb300 import configs, fp8
from compressed_kv_sparse_compressor_gb300.layer import DeviceLayer
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_example_of_the_8_bit_layer():
    require_gpu()
    code = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "set_weights_quant" in b]
    assert len(code) == 1
    T = 70
    shape = configs.LayerShape(d_model=520, head_dim=128, n_rot=64, idx_head_dim=64, n_heads=8, ratio=4, top_k=8,
                               dtype="f32", w_std=0.04)
    g = torch.Generator(device="cuda").manual_seed(11)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")
    lanes = [configs.lane_weights(shape, 5, 0, lane, device="cuda", gamma_std=0.1) for lane in ("attn", "idx")]
    names = dict(zip(("wkv", "wgate", "ape", "norm"), lanes[0]))
    names.update(zip(("wkv_idx", "wgate_idx", "ape_idx", "norm_idx"), lanes[1]))
    names.update(shape=shape, comp_cap=T, idx_cap=T, x=randn(T, 520), res=randn(T, 520), gain=1 + 0.1 * randn(520), pos0=0,
                 wq=0.02 * randn(96, 520))
    want_h = names["x"] + names["res"]
    exec(code[0], names)
    layer = names["layer"]
    layer.sync()
    assert torch.equal(names["res"], want_h)
    rows = ref.values(names["q"].view(torch.uint8), names["scale"], 1)
    # the same rows through the float layer, on the values that the codes stand for
    plain = DeviceLayer(shape, T, T)
    plain.state_init()
    plain.set_weights(*[[ref.values(t.q.view(torch.uint8), t.scale, 128).float() for t in map(fp8.quantize_weight, w[:2])] +
                        list(w[2:]) for w in lanes])
    plain.compress_prefill(rows.float().contiguous(), 0)
    plain.sync()
    for name in ("attn_kv", "attn_score", "idx_kv", "idx_score", "idx_comp"):
        u, v = getattr(plain, name), getattr(layer, name)
        fin = torch.isfinite(u)
        assert torch.equal(fin, torch.isfinite(v)), name
        # the path's tolerance for float-accumulated values
        assert ((u - v)[fin].abs() <= 1e-4 + 2e-3 * u[fin].abs()).all(), name
    # the first window's row pools its own four tokens alone: what the frontier held before must not count.  The rows
    # went through E4M3 (2^-4 of a value half a step, in blocks whose scale may differ by one): two steps
    a, b = plain.attn_comp[0, :T // 4], layer.attn_comp[0, :T // 4]
    assert ((a - b).abs() <= 2 * 2.0 ** -3 * a.abs().amax(1, keepdim=True)).all()
    w = fp8.quantize_weight(names["wq"])
    want = rows @ ref.values(w.q.view(torch.uint8), w.scale, 128).T
    mag = rows.abs() @ ref.values(w.q.view(torch.uint8), w.scale, 128).abs().T
    assert ((names["out"][0].double() - want).abs() <= 520 * 2.0 ** -23 * mag).all()
