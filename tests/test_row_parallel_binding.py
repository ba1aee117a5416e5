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


# -------------------------------------------------------------------------------- sizes past an int
def cuda_tensor(shape, dtype, stride=None):
    """A tensor that says it lies on a GPU, of any size, without memory: the binding's own view of it."""
    import torch

    dense = stride is None

    class OnGpu(torch.Tensor):
        def data_ptr(self):
            return 0x10000

        def is_contiguous(self):
            return dense

        def get_device(self):
            return 0

        __torch_function__ = torch._C._disabled_torch_function_impl

        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise NotImplementedError(func)

    if dense:
        stride, n = [], 1
        for d in reversed(shape):
            stride.insert(0, n)
            n *= d
    return torch.Tensor._make_wrapper_subclass(OnGpu, shape, strides=stride, dtype=dtype, device="cuda:0")


BIG = 1 << 32


def past_an_int():
    import torch

    import bit_tensor_activation_b200 as hq

    bf, i8, f32, i32, u8 = torch.bfloat16, torch.int8, torch.float32, torch.int32, torch.uint8
    t = cuda_tensor

    def product(P=1, T=4, H=64, K=64, lda=None, ldo=None):
        lda, ldo = lda or K, ldo or H
        return lambda: hq.hq_int8_matmul(t((P, T, K), i8, (T * lda, lda, 1)), t((P, T), f32), t((P, H, K), i8), t((P, H), f32),
                                         t((P, T, H), bf, (T * ldo, ldo, 1)))

    def tokens(rows=4, K=64, ldx=None, ldq=None):
        return lambda: hq.hq_quantize_tokens(t((rows, K), bf, (ldx or K, 1)), t((rows, K), i8, (ldq or K, 1)), t((rows,), f32))

    def pack(T=4, K=64, H=64, k=8, lda=None):
        lda = lda or K
        return lambda: hq.hq_int8_matmul_pack(t((1, T, K), i8, (T * lda, lda, 1)), t((1, T), f32), t((1, H, K), i8), t((1, H), f32),
                                              t((k,), i32), t((H - k,), i32), t((1, H), f32), t((1, H), u8),
                                              t((1, T, (H - k) // 8), i32), t((1, k, T), bf))

    def norm(T=4, H=64, ldq=None, **kw):
        x = t((T, H), bf)
        return lambda: hq.hq_residual_norm(x, x, x, h=x, q=t((T, H), i8, (ldq or H, 1)), q_scale=t((T,), f32), **kw)

    return {"as it is: tokens": (tokens(), None), "as it is: product": (product(), None), "as it is: pack": (pack(), None),
            "as it is: norm": (norm(), None),
            "tokens, K": (tokens(K=BIG + 64), "K|pitch"), "tokens, x's pitch": (tokens(ldx=BIG + 64), "pitch"),
            "tokens, q's pitch": (tokens(ldq=BIG + 64), "pitch"), "product, T": (product(T=BIG + 4), "T"),
            "product, K": (product(K=BIG + 64), "K|pitch"), "product, H": (product(H=BIG + 64), "H|pitch"),
            "product, a's pitch": (product(lda=BIG + 64), "pitch"), "product, out's pitch": (product(ldo=BIG + 64), "pitch"),
            "pack, T": (pack(T=BIG + 4), "T"), "pack, a's pitch": (pack(lda=BIG + 64), "pitch"),
            "norm, T": (norm(T=BIG + 4), "T"), "norm, H": (norm(H=BIG + 64), "H|pitch"),
            "norm, q's pitch": (norm(ldq=BIG + 64), "pitch"), "norm, post": (norm(post=BIG + 1), "post"),
            "norm, pre": (norm(pre=BIG + 1), "pre")}


CASES = ["as it is: tokens", "as it is: product", "as it is: pack", "as it is: norm", "tokens, K", "tokens, x's pitch",
         "tokens, q's pitch", "product, T", "product, K", "product, H", "product, a's pitch", "product, out's pitch", "pack, T",
         "pack, a's pitch", "norm, T", "norm, H", "norm, q's pitch", "norm, post", "norm, pre"]


@pytest.mark.parametrize("case", CASES)
def test_what_an_int_does_not_hold_is_refused(case, monkeypatch):
    """2^32 more than a size that fits is the same 32 bits: cut to them, the call would read another tensor."""
    import bit_tensor_activation_b200 as hq

    reached = []
    monkeypatch.setattr(hq, "_call", lambda fn, where, *args: reached.append(where))
    call, match = past_an_int()[case]
    if match is None:
        call()
        assert len(reached) == 1
        return
    with pytest.raises(ValueError, match=match):
        call()
    assert not reached
