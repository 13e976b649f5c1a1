"""The package in another folder: without _ssu_torch.so, and with its own libraries."""
import os
import shutil
import subprocess
import sys

import mamba_selective_state_amd as ssu

PACKAGE = os.path.dirname(os.path.abspath(ssu.__file__))


def copy_package(to, without=()):
    dst = os.path.join(str(to), os.path.basename(PACKAGE))
    os.mkdir(dst)
    for name in os.listdir(PACKAGE):
        if name.endswith((".py", ".so")) and name not in without:
            shutil.copy(os.path.join(PACKAGE, name), dst)
    return dst


def run(folder, code):
    r = subprocess.run([sys.executable, "-c", code], cwd=str(folder), capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(folder)})
    assert r.returncode == 0, r.stderr
    return r.stdout.split()


def test_without_the_torch_module(tmp_path):
    """The state operators and the layer operators' C entry points need libssu.so alone; a call of
    the three functions that are in the module says that it is missing."""
    copy_package(tmp_path, without=("_ssu_torch.so",))
    out = run(tmp_path, """
import torch
import mamba_selective_state_amd as ssu
print(ssu.__file__)
assert ssu.ssu_abi_version() > 0 and callable(ssu.selective_state_update)
assert ssu.ssu_mx_linear_workspace_bytes(ssu.SsuMxLinearArgs()) == 0
x = torch.zeros(2, 64)
for f in (lambda: ssu.add_rms_norm(x, x[0]), lambda: ssu.mx_linear(x, x, x), lambda: ssu.token_logprobs(x, x[:, 0])):
    try:
        f()
    except ImportError as e:
        assert "_ssu_torch" in str(e), e
        print("refused")
""")
    assert out[0].startswith(str(tmp_path)) and out[1:] == ["refused"] * 3


def test_copied_package_uses_its_own_library(tmp_path):
    dst = copy_package(tmp_path)
    out = run(tmp_path, """
import torch
import mamba_selective_state_amd as ssu
try:
    ssu.add_rms_norm(torch.zeros(2, 64), torch.zeros(64))
except ValueError:
    pass
print(*sorted({l.split()[-1] for l in open("/proc/self/maps") if "ssu" in l and ".so" in l}))
""")
    assert out == [os.path.join(dst, n) for n in ("_ssu_torch.so", "libssu.so")]
