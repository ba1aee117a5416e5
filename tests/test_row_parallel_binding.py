"""The Python binding without a GPU: what it does where its C++ module does not load, and sizes that an int of
the C ABI cannot hold."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "bit_tensor_activation_b200"
PROGRAM = r"""
import warnings
import torch
{before}
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import bit_tensor_activation_b200 as hq
    from bit_tensor_activation_b200 import exchange
said = [str(w.message) for w in said if issubclass(w.category, RuntimeWarning)]
assert hq.hq_wire_bytes_per_row(64, 8) > 0 and hq.hq_status_string(0) == "HQ_OK"
x, q, s = torch.zeros(4, 64).bfloat16(), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
for call in (lambda: hq.hq_quantize_tokens(x, q, s), lambda: hq.hq_residual_norm(x, x, x, h=x),
             lambda: hq.hq_int8_matmul(q[None], s[None], q[None], s[None], x[None]),
             lambda: hq.hq_dequant_reduce(q.int()[None], x[None], s.int(), s.int(), s[None], s[None], x)):
    try:
        call()
        raise SystemExit("not refused")
    except (TypeError, ValueError):
        pass
print(len(said), "built" if "do not load" not in "".join(said) else "none", said)
"""


def import_copy(tmp_path, module, before=""):
    """The package, copied, with `module` in the place of the C++ module (None: nothing there)."""
    to = tmp_path / NAME
    to.mkdir()
    src = os.path.join(ROOT, NAME)
    for n in ("__init__.py", "exchange.py"):
        shutil.copy(os.path.join(src, n), to / n)
    os.symlink(os.path.join(src, "libhq.so"), to / "libhq.so")
    if module is not None:
        if isinstance(module, bytes):
            (to / "_hqargs.so").write_bytes(module)
        else:
            shutil.copy(module, to / "_hqargs.so")
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(before=before)], cwd=tmp_path, text=True, capture_output=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.strip()


@pytest.mark.parametrize("module", [None, b"not a library"], ids=["missing", "broken"])
def test_the_library_alone_is_enough(tmp_path, module):
    assert import_copy(tmp_path, module).startswith("1 none")


def test_a_module_of_another_torch_is_not_used(tmp_path):
    built = os.path.join(ROOT, NAME, "_hqargs.so")
    for v in ("0.0.1", "torch.__version__.split('+')[0] + '0'"):
        sub = tmp_path / str(len(v))
        sub.mkdir()
        said = import_copy(sub, built, "torch.__version__ = " + (v if "torch" in v else repr(v)))
        assert said.startswith("1 none") and "was built for torch" in said


def test_the_built_module_loads(tmp_path):
    assert import_copy(tmp_path, os.path.join(ROOT, NAME, "_hqargs.so")).startswith("0 built")
