"""DecoupledLayer makes its device current around its calls: the attention's own run on the current one, the layer operators on
their tensors' (no GPU needed: the calls and torch's device context are recorded)."""
import types

import pytest
import torch

import block_sparse_cluster_b200 as da
from block_sparse_cluster_b200 import layer as module


@pytest.mark.parametrize("call", ["prepare", "project", "attend", "step", "status"])
def test_every_call_runs_on_the_layers_device(call, monkeypatch):
    current, seen = [], []

    class Current:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *exc):
            current.pop()

    def noted(name):
        return lambda *a, **kw: seen.append((name, current[-1] if current else None))
    monkeypatch.setattr(torch.cuda, "device", Current)
    for name in ("da_rms_norm_i8", "da_linear_i8", "da_rope", "da_quantize_i8"):
        monkeypatch.setattr(module, name, noted(name))
    layer = da.DecoupledLayer.__new__(da.DecoupledLayer)
    layer.dims, layer.width, layer.rope, layer.eps = da.Dims(1, 2, 4, 64, 64, 64), 8, da.Rope((32, 16, 16), (1, 2, 2)), 1e-6
    layer.weights = da.LayerWeights(None, (None, None), (None, None), (None, None))
    layer.engine = types.SimpleNamespace(ws=None, **{n: noted("engine." + n) for n in ("prepare", "step", "status")})
    where = torch.device("meta")
    layer.Q, layer.K, layer.V, layer.O = (torch.empty(1, 2, 4, 64, device=where) for _ in range(4))
    layer._qk = torch.empty(4, 256, device=where)
    layer._x = layer._x_scale = layer._o = layer._o_scale = torch.empty(1, device=where)
    x = torch.empty(1, 4, 8, device=where)
    arguments = dict(prepare=(None, None), project=(x,), attend=(None, x), step=(x, None, x), status=())[call]
    getattr(layer, call)(*arguments)
    assert len(seen) >= 1 and not current
    assert all(device == where for _, device in seen), seen
