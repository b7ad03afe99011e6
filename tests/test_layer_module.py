"""The attention does not hang on the layer operators' marshalling module loading: one built for another torch costs the layer
operators alone, loudly (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import block_sparse_cluster_b200 as da

SCRIPT = """
import block_sparse_cluster_b200 as da
import torch
assert da.da_version() > 0 and da.da_workspace_bytes(da.Dims(1, 1, 256, 64, 64, 128)) > 0
x, q, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
h = x.view(1, 1, 4, 64)
for call in (lambda: da.da_rms_norm(x, None, x), lambda: da.da_rms_norm_i8(x, None, q, s), lambda: da.da_quantize_i8(x, q, s),
             lambda: da.da_linear_i8(q, s, q, s, x[:, :4], q), lambda: da.da_rope(h, h, da.Rope((32, 16, 16)))):
    try:
        call()
    except ImportError as e:
        assert "_layer_call.so does not load" in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


def test_attention_is_there_when_the_marshalling_module_does_not_load(tmp_path):
    src = os.path.dirname(da.LIB_PATH)
    pkg = tmp_path / "block_sparse_cluster_b200"
    pkg.mkdir()
    for name in ("__init__.py", "layer.py", "libda.so"):
        shutil.copy(os.path.join(src, name), pkg / name)
    (pkg / "_layer_call.so").write_bytes(b"no shared object")
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr


def test_lazily_negated_tensors_are_refused():
    """torch keeps the imaginary part of a conjugate as the memory of the plain one and a mark to negate it, which no call here reads."""
    import pytest
    import torch
    x = torch.randn(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    lazy = torch.complex(x, x).conj().imag
    assert lazy.is_neg()
    h, r = lazy.reshape(1, 1, 4, 64), da.Rope((32, 16, 16), (1, 2, 2))
    plain = x.view(1, 1, 4, 64)
    for call in (lambda: da.da_rms_norm(lazy, None, x), lambda: da.da_rms_norm(x, None, x, residual=lazy), lambda: da.da_rms_norm_i8(lazy, None, q, s),
                 lambda: da.da_rms_norm(x, lazy[0], x), lambda: da.da_quantize_i8(lazy, q, s), lambda: da.da_linear_i8(q, lazy[:, 0], q, s, x[:, :4], q),
                 lambda: da.da_rope(torch._neg_view(plain), plain, r), lambda: da.da_rope(plain, torch._neg_view(plain), r)):
        with pytest.raises(da.DAError, match="negated"):
            call()
