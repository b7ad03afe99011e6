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
