"""Empty tensors of any other dimensions: the statistics' size, N * groups, must not wrap
around in the overlap checks.  In a process without a device: a call that passes the
checks ends in the runtime's first call, EP_ERR_CUDA, or returns EP_OK without any."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import ctypes, json, sys
sys.path.insert(0, %r)
from transformer_epilogue_gb300 import _binding
lib = _binding.load_library()
A, B, C, D, E, F, G, H, I, J = (0x7F0000000000 + i * (1 << 36) for i in range(10))
out = []
for shape, groups in (((1 << 59, 0, 8), 2), ((1 << 60, 0, 8), 2), ((1 << 61, 0, 8), 8), ((5, 0, 8), 2), ((0, 1 << 50, 8), 4)):
    s = (ctypes.c_int64 * 3)(*shape)
    for dg, db in ((H, I), (B, I), (H, None), (None, None)):
        out.append([shape, lib.ep_group_norm_grad(1, A, J, s, C, D, groups, 0, E, F, G, dg, db, None, 0, None)])
    out.append([shape, lib.ep_group_norm(1, A, s, B, C, groups, 1e-5, 0, D, E, F, None, 0, None)])
print(json.dumps(out))
"""


def test_empty_tensors_pass_the_overlap_checks():
    from transformer_epilogue_gb300 import build
    build.build()
    p = subprocess.run([sys.executable, "-c", CODE % ROOT], env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                       capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert p.returncode == 0, p.stderr[-2000:]
    got = json.loads(p.stdout)
    assert len(got) == 25
    for k, (shape, status) in enumerate(got):
        assert status == (4 if k % 5 < 3 else 0), (shape, k % 5, status)
