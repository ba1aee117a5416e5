"""The row-parallel calls without a GPU: what the C ABI and the binding refuse, and the rounding that
a token's codes rest on."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import bit_tensor_activation_b200 as hq

A = 0x10000  # never dereferenced: every call below fails its checks first
MIS = A + 4


def c(p):
    return ctypes.c_void_p(p)


def quantize(x=A, ldx=64, rows=4, K=64, q=A, ldq=64, scale=A):
    return hq.lib().hq_quantize_tokens(c(x), ldx, rows, K, c(q), ldq, c(scale), None)


def matmul(a=A, lda=64, a_s=A, w=A, ldw=64, w_s=A, bias=0, P=2, T=4, H=64, K=64, out=A, ldo=64, odt=0):
    return hq.lib().hq_int8_matmul(c(a), lda, c(a_s), c(w), ldw, c(w_s), c(bias), P, T, H, K, c(out), ldo, odt, None)


def pack(a=A, lda=64, a_s=A, w=A, ldw=64, w_s=A, P=2, T=4, H=64, K=64, k=8, keep=A, rest=A, inv=A, z=A, codes=A,
         side=A):
    return hq.lib().hq_int8_matmul_pack(c(a), lda, c(a_s), c(w), ldw, c(w_s), P, T, H, K, k, c(keep), c(rest), c(inv),
                                        c(z), c(codes), c(side), None)


def norm(y=A, ydt=0, res=A, out=A, rdt=0, T=4, H=64, post=0, post_w=0, gate=0, gate_rows=1, alpha=1.0, beta=1.0, pre=1,
         pre_w=0, eps=1e-6, h=A, q=0, ldq=64, q_s=0):
    f = ctypes.c_float
    return hq.lib().hq_residual_norm(c(y), ydt, c(res), c(out), rdt, T, H, post, c(post_w), None, c(gate), gate_rows,
                                     f(alpha), f(beta), pre, c(pre_w), None, f(eps), c(h), c(q), ldq, c(q_s), None)


@pytest.mark.parametrize("call,kw,status", [
    (quantize, dict(rows=-1), 1), (quantize, dict(rows=1 << 31), 1), (quantize, dict(K=0), 1),
    (quantize, dict(K=65537, ldx=65544, ldq=65552), 1), (quantize, dict(ldx=63), 1), (quantize, dict(ldx=68), 1),
    (quantize, dict(ldq=48), 1), (quantize, dict(ldq=72), 1), (quantize, dict(x=0), 1), (quantize, dict(q=0), 1),
    (quantize, dict(scale=0), 1), (quantize, dict(x=MIS), 2), (quantize, dict(q=MIS), 2), (quantize, dict(scale=A + 2), 2),
    (quantize, dict(rows=0), 0), (quantize, dict(rows=0, x=0, q=0, scale=0), 0),
    (matmul, dict(P=0), 1), (matmul, dict(P=65), 1), (matmul, dict(T=-1), 1), (matmul, dict(H=0), 1),
    (matmul, dict(H=60), 1), (matmul, dict(H=1048584, ldo=1048584), 1), (matmul, dict(K=0), 1), (matmul, dict(K=65), 1),
    (matmul, dict(K=65537, lda=65552, ldw=65552), 1), (matmul, dict(lda=72), 1), (matmul, dict(ldw=72), 1),
    (matmul, dict(ldo=56), 1), (matmul, dict(ldo=68), 1), (matmul, dict(odt=2), 1), (matmul, dict(a=0), 1),
    (matmul, dict(a_s=0), 1), (matmul, dict(w=0), 1), (matmul, dict(w_s=0), 1), (matmul, dict(out=0), 1),
    (matmul, dict(a=A + 8), 2), (matmul, dict(w=A + 8), 2), (matmul, dict(w_s=MIS), 2), (matmul, dict(bias=A + 2), 2),
    (matmul, dict(out=A + 8), 2), (matmul, dict(a_s=A + 2), 2), (matmul, dict(T=0), 0),
    (matmul, dict(T=0, a=0, a_s=0, out=0), 0),
    (pack, dict(P=65), 1), (pack, dict(H=32776), 1), (pack, dict(k=4), 1), (pack, dict(k=72), 1), (pack, dict(keep=0), 1),
    (pack, dict(rest=0), 1), (pack, dict(inv=0), 1), (pack, dict(z=0), 1), (pack, dict(codes=0), 1),
    (pack, dict(side=0), 1), (pack, dict(inv=MIS), 2), (pack, dict(z=A + 8), 2), (pack, dict(side=MIS), 2),
    (pack, dict(codes=A + 2), 2), (pack, dict(keep=A + 2), 2), (pack, dict(T=0), 0),
    (pack, dict(T=0, k=0, keep=0, side=0, codes=0), 0), (pack, dict(T=0, k=64, rest=0, side=0, codes=0), 0),
    (norm, dict(T=-1), 1), (norm, dict(H=12), 1), (norm, dict(H=32776), 1), (norm, dict(ydt=2), 1), (norm, dict(rdt=-1), 1),
    (norm, dict(post=3), 1), (norm, dict(pre=-1), 1), (norm, dict(pre=0), 1), (norm, dict(h=0), 1),
    (norm, dict(eps=-1.0), 1), (norm, dict(eps=float("nan")), 1), (norm, dict(alpha=float("inf")), 1),
    (norm, dict(beta=float("nan")), 1), (norm, dict(gate=A, gate_rows=0), 1), (norm, dict(q=A), 1), (norm, dict(q_s=A), 1),
    (norm, dict(q=A, q_s=A, ldq=72), 1), (norm, dict(q=A, q_s=A, ldq=48), 1), (norm, dict(y=0), 1), (norm, dict(res=0), 1),
    (norm, dict(out=0), 1), (norm, dict(y=MIS), 2), (norm, dict(gate=MIS), 2), (norm, dict(pre_w=MIS), 2),
    (norm, dict(h=A + 8), 2), (norm, dict(q=A + 8, q_s=A), 2), (norm, dict(q=A, q_s=A + 2), 2), (norm, dict(T=0), 0),
])
def test_host_checks(call, kw, status):
    assert call(**kw) == status


def test_the_binding_refuses_tensors_of_the_host():
    import torch

    x, q, s = torch.zeros(4, 64).bfloat16(), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(TypeError):
        hq.hq_quantize_tokens(x, q, s)
    with pytest.raises(TypeError):
        hq.hq_int8_matmul(q[None], s[None], q[None], s[None], x[None])
    with pytest.raises(TypeError):
        hq.hq_residual_norm(x, x, x, h=x)


def test_tensors_without_storage_are_refused_not_fatal():
    """A fake tensor throws in C++ when it is asked for its address; the binding says what is wrong."""
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode():
        x, q, s = (torch.empty(4, 64, dtype=torch.bfloat16), torch.empty(4, 64, dtype=torch.int8), torch.empty(4))
        with pytest.raises(TypeError):
            hq.hq_quantize_tokens(x, q, s)
    with pytest.raises(TypeError):
        hq.hq_int8_matmul(None, None, None, None, None)
    with pytest.raises((TypeError, AttributeError)):
        hq.hq_residual_norm(torch.zeros(4, 64, dtype=torch.bfloat16, device="meta"), None, None)


def half_even(f: Fraction) -> int:
    return round(f)  # Python rounds a Fraction's half to even


def kernel_code(x, amax):
    """The kernel's steps in numpy's fp32: product, 20 significant bits, rounding to an integer."""
    inv = np.float32(127.0) / np.float32(amax)
    t = (np.float32(x) * inv).view(np.uint32)
    t = np.uint32((int(t) + 8) & 0xFFFFFFF0).view(np.float32)
    return int(np.rint(t))


def test_a_code_is_the_exact_quotients_rounding():
    """Every pair of bf16 significands, at every distance of exponents where the quotient is not far
    below one half: the codes are rint(127 x / amax) of the exact quotient, its ties to even."""
    m = np.arange(128, 256, dtype=np.float32)
    for d in range(0, 10):
        x, amax = np.meshgrid(m, m * np.float32(2.0) ** d)
        ok = x <= amax
        x, amax = x[ok], amax[ok]
        t = ((x * (np.float32(127.0) / amax)).view(np.uint32) + np.uint32(8)) & np.uint32(0xFFFFFFF0)
        got = np.rint(t.view(np.float32)).astype(np.int64)
        n, den = 127 * x.astype(np.int64), amax.astype(np.int64)  # exact integers
        twice = 2 * n
        lo = (twice + den) // (2 * den)  # floor(q + 1/2)
        tie = (twice + den) % (2 * den) == 0
        want = np.where(tie & (lo % 2 == 1), lo - 1, lo)
        assert np.array_equal(got, want), d
    for x, amax in ((1.0, 2.0), (64.0, 128.0), (127.0, 254.0), (0.0, 1.0)):
        assert kernel_code(x, amax) == half_even(Fraction(127) * Fraction(x) / Fraction(amax))
