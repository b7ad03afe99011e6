"""The layer operators run together around the attention, as DecoupledLayer runs them: every stage against
the fp64 oracle on the values the stage before left on the GPU, so that no stage hides behind another's
rounding.  Tolerances are those of the operators' own tests and of the attention parity tests."""
import numpy as np
import pytest
import torch

import block_sparse_cluster_b200 as da
import oracle
import workloads as W
from tests import parity as P
from tests.test_gpu_layer import _close, _half, _linear_close, _rope_check

pytestmark = pytest.mark.gpu


def _layer(w, width, norms, seed):
    g = torch.Generator().manual_seed(seed)
    dims = P.dims_of(w)
    dt, hd = w.torch_dtype, w.H * w.d

    def weight(rows, cols):
        return (torch.randn(rows, cols, generator=g) / cols ** 0.5).to(dt).cuda()
    n = {"head": w.d, "full": hd}.get(norms)
    norm = None if n is None else (1 + 0.1 * torch.randn(n, generator=g)).to(dt).cuda()
    weights = da.LayerWeights.quantize((1 + 0.1 * torch.randn(width, generator=g)).to(dt).cuda(), weight(hd, width), weight(hd, width),
                                       weight(hd, width), weight(width, hd), q_norm=norm, k_norm=norm,
                                       v_bias=torch.randn(hd, generator=g).cuda(), out_bias=torch.randn(width, generator=g).cuda())
    axes = (44, 42, 42) if w.d == 128 else (20, 22, 22)
    layer = da.DecoupledLayer(dims, width, weights, da.Rope(axes=axes, grid=(w.T, w.Hs, w.Ws)))
    x = torch.randn(w.B, w.N, width, generator=g).to(dt)
    r = torch.randn(w.B, w.N, width, generator=g).to(dt)
    return dims, layer, x, r


@pytest.mark.parametrize("name,width,norms,residual", [
    ("tiny", 200, "head", True), ("tiny", 128, "full", False), ("wan13b", 256, "full", True), ("wan13b", 1001, None, True),
])
def test_layer_stages(name, width, norms, residual):
    w = W.WORKLOADS["tiny"] if name == "tiny" else W.scaled(W.WORKLOADS["wan13b"], H=2, T=1)
    if name == "tiny" and residual:
        w = W.scaled(w, B=2, T=2)
    dims, layer, x, r = _layer(w, width, norms, seed=len(name) + width)
    inp = W.make_inputs(w, seed=3)
    layer.prepare(inp.kv_idx.cuda(), inp.kv_cnt.cuda())
    xc, rc = x.cuda(), r.cuda() if residual else None
    layer.project(xc, rc)
    assert torch.equal(xc.cpu(), x)
    B, H, N, d = w.B, w.H, w.N, w.d
    rows = x.reshape(B * N, width)
    if residual:
        total = (x.double() + r.double()).numpy()
        _close(rc, total, np.abs(total) * (_half(w.torch_dtype) + 2.0 ** -23))
    q, scale, _ = oracle.rms_norm_i8(rows, r.reshape(B * N, width) if residual else None, layer.weights.norm, layer.eps)
    assert np.array_equal(layer._x.cpu().numpy().astype(np.int64), q)
    _close(layer._x_scale, scale, scale * 2.0 ** -19)
    codes, scales = layer.weights.qk
    _linear_close(layer._qk, layer._x, layer._x_scale.cpu(), codes, scales.cpu(), None, w.torch_dtype)
    codes, scales = layer.weights.v
    _linear_close(layer.V.permute(0, 2, 1, 3).reshape(B * N, H * d), layer._x, layer._x_scale.cpu(), codes, scales.cpu(),
                  layer.weights.v_bias.cpu(), w.torch_dtype)
    slots = layer._qk.view(B, N, 2, H, d)
    for slot, out in ((0, layer.Q), (1, layer.K)):
        _rope_check(slots[:, :, slot].permute(0, 2, 1, 3), out, layer.rope, None, layer.weights.q_norm, layer.eps, w.torch_dtype)

    # initial clustering of the projected keys, then the attention and the output projection
    cent = layer.K[:, :, :w.C].contiguous()
    da.kmeans(dims, layer.K, cent, 2, layer.engine.stats, layer.engine.ws)
    out = torch.empty_like(xc)
    layer.attend(cent, out)
    assert layer.status() == 0
    got = W.Inputs(w, 0, layer.Q.cpu(), layer.K.cpu(), layer.V.cpu(), cent.cpu(), inp.kv_idx, inp.kv_cnt, inp.plans)
    for b in range(B):
        a = layer.engine.stats.assign[b, 0].cpu().numpy().astype(np.int64)
        P.check_assignment(got, b, 0, a)
        ref = oracle.attention_qblock(got.Q[b, 0], got.K[b, 0], got.V[b, 0], got.centroids[b, 0], got.plans[b][0][1], a, 1, w.block)
        o = layer.O[b, 0, w.block:2 * w.block].float().cpu().numpy()
        assert np.abs(o - ref).max() <= P.ATT_TOL[w.dtype] * max(1.0, np.abs(got.V[b, 0].float().numpy()).max() / 4)
    q, m = oracle.row_codes(layer.O.cpu().permute(0, 2, 1, 3).reshape(B * N, H * d))
    assert np.array_equal(layer._o.cpu().numpy().astype(np.int64), q)
    codes, scales = layer.weights.out
    _linear_close(out.view(B * N, width), layer._o, layer._o_scale.cpu(), codes, scales.cpu(), layer.weights.out_bias.cpu(), w.torch_dtype)

    # the whole step at once, on a stream of its own, gives the same bits
    again, r2 = torch.zeros_like(out), r.cuda() if residual else None
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    layer.step(xc, cent, again, residual=r2, stream=side)
    side.synchronize()
    assert layer.status(side) == 0 and torch.equal(again, out) and (not residual or torch.equal(r2, rc))


def test_layer_refuses_weights_of_another_shape():
    w = W.WORKLOADS["tiny"]
    dims = P.dims_of(w)
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(da.DAError):
        da.DecoupledLayer(dims, 64, da.LayerWeights(None, q, q, q), da.Rope((32, 16, 16), (4, 16, 16)))
