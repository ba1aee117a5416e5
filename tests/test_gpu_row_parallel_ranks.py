"""The row-parallel layer through the exchange module, and the give-up paths of its kernels.

Ranks are played one after another on one GPU, the buffers moved as the collective would move them; no
kernel waits for another rank.  The pipelines' waits are made to run out as in the compression's own
kernels: producers delayed well past a short bound on the consumers, which give up, record
HQ_ERR_TIMEOUT and leave the context usable.
"""
import pytest
import torch

import bit_tensor_activation_b200 as hq
from bit_tensor_activation_b200 import exchange as ex
from gpu_helpers import DEV, assert_no_device_error
from test_gpu_row_parallel import (BF, D, close, gen, operands, pitched, plain_norm, plain_product, plain_tokens, same,
                                   selection, up)

pytestmark = pytest.mark.gpu


def setup(P, T, H, K, k, seed=5):
    """Activations of every rank, weights in the features' order, and shared parameters."""
    a, a_s, w, w_s = operands(seed, P, T, H, K)
    x = pitched((a.float() * a_s[..., None]).to(BF), up(K, 8))[0]
    keep, rest, zero = selection(seed, P, H, k)
    scale = torch.full((P, H), 0.25, device=DEV) * float(a_s.mean() * w_s.mean()) * 127 * 64 * K ** 0.5
    params = ex.HybridParams(keep, rest, scale, (1 / scale).contiguous(), zero)
    return x, w, w_s, params


def plain_sum(x, w, w_s, p):
    """quantize-pack of the plain product, and the reduction."""
    q, s = plain_tokens(x)
    part = plain_product(q, s, w, w_s).to(BF)
    P, T, H = part.shape
    k = p.k
    codes = torch.empty(P, T, (H - k) // 8, dtype=torch.int32, device=DEV)
    side = torch.empty(P, k, T, dtype=BF, device=DEV)
    hq.hq_quantize_pack(part, p.keep_idx, p.rest_idx, p.inv_scale, p.zero, codes, side)
    out = torch.empty(T, H, dtype=BF, device=DEV)
    hq.hq_dequant_reduce(codes, side, p.keep_idx, p.rest_idx, p.scale, p.zero, out)
    return out


@pytest.mark.parametrize("T,K", [(4, 40), (128, 264), (400, 128)])
@pytest.mark.parametrize("scheme", ["allgather", "reduce_scatter"])
def test_layer_through_the_all_reduce(scheme, T, K):
    P, H, k = 4, 528, 16
    x, w, w_s, p = setup(P, T, H, K, k)
    want = plain_sum(x, w, w_s, p)
    layers = [ex.Int8RowParallel(ex.HybridAllReduce(p, T, r, scheme), w[r], w_s[r]) for r in range(P)]
    wires = [layer.wire(x[r]) for r, layer in enumerate(layers)]
    res = torch.randn(T, H, generator=gen(1), device=DEV).to(BF)
    for j, layer in enumerate(layers):
        if scheme == "allgather":
            total = layer.reducer.reduce_block(torch.cat([c for c, _ in wires]), torch.cat([s for _, s in wires]))
            same(total, want, f"rank {j}")
        else:
            rows = slice(j * T // P, (j + 1) * T // P)
            block = layer.reducer.reduce_block(torch.stack([c[j] for c, _ in wires]), torch.stack([s[j] for _, s in wires]))
            same(block, want[rows], f"rank {j}'s block")
            total = want
        r = res.clone()
        q, s = layer.finish(total, r, post=hq.HQ_NORM_RMS)
        u, mag = plain_norm(total, hq.HQ_NORM_RMS, None, None, 1e-6)
        exact = res.to(D) + u
        close(r, exact, res.to(D).abs() + u.abs() + mag, "residual")
        n, _ = plain_norm(r, hq.HQ_NORM_RMS, None, None, 1e-6)
        off = (q.to(D) * s.to(D)[:, None] - n).abs()
        # half a code's step, and the bf16 rounding of the norm before it
        assert (off <= s.to(D)[:, None] * 0.5 * (1 + 1e-5) + n.abs() * (2.0 ** -8 + 1e-5)).all()
    assert_no_device_error()


def test_layer_through_the_peers_wires():
    P, T, H, K, k = 3, 50, 544, 100, 32
    x, w, w_s, p = setup(P, T, H, K, k, seed=6)
    wires = [(torch.empty(T, (H - k) // 8, dtype=torch.int32, device=DEV), torch.empty(k, T, dtype=BF, device=DEV))
             for _ in range(P)]
    layers = [ex.Int8RowParallel(ex.PeerAllReduce(p, T, r, wires), w[r], w_s[r]) for r in range(P)]
    for r, layer in enumerate(layers):
        layer.wire(x[r])
    want = plain_sum(x, w, w_s, p)
    for layer in layers:
        same(layer.reducer.reduce(), want, "sum")
    same(layers[-1](x[-1]), want, "the whole call of the last rank")
    assert_no_device_error()


LIMIT, DELAY = 20_000, 100_000_000  # cycles: about 10 us, and 50 ms


@pytest.mark.parametrize("what", ["pair", "pair wire", "few", "few of a cluster", "norm"])
def test_waits_that_run_out(what):
    if what == "norm":
        T, H = 1200, 8192
        y, res = torch.randn(T, H, device=DEV).to(BF), torch.randn(T, H, device=DEV).to(BF)
        out, h = torch.empty_like(res), torch.empty_like(res)
        call = lambda: hq.hq_residual_norm(y, res, out, h=h)  # noqa: E731
        check = lambda: close(out, res.to(D) + y.to(D), res.to(D).abs() + y.to(D).abs(), "residual")  # noqa: E731
    else:
        P, T, H, K = {"pair": (2, 600, 1024, 1500), "pair wire": (1, 300, 512, 256), "few": (8, 20, 8192, 600),
                      "few of a cluster": (1, 9, 512, 2048)}[what]
        a, a_s, w, w_s = operands(3, P, T, H, K)
        if what == "pair wire":
            keep, rest, zero = selection(2, P, H, 8)
            inv = torch.full((P, H), 1e-2, device=DEV)
            order = torch.cat([rest, keep]).long()
            wo, so = w[:, order].contiguous(), w_s[:, order].contiguous()
            codes, side = torch.empty(P, T, (H - 8) // 8, dtype=torch.int32, device=DEV), torch.empty(P, 8, T, dtype=BF, device=DEV)
            want = torch.empty_like(codes), torch.empty_like(side)
            hq.hq_quantize_pack(plain_product(a, a_s, w, w_s).to(BF), keep, rest, inv, zero, *want)
            call = lambda: hq.hq_int8_matmul_pack(a, a_s, wo, so, keep, rest, inv, zero, codes, side)  # noqa: E731
            check = lambda: (same(codes, want[0], "codes"), same(side, want[1], "side"))  # noqa: E731
        else:
            out = torch.empty(P, T, H, dtype=BF, device=DEV)
            call = lambda: hq.hq_int8_matmul(a, a_s, w, w_s, out)  # noqa: E731
            check = lambda: same(out, plain_product(a, a_s, w, w_s).to(BF), "out")  # noqa: E731
    assert_no_device_error()
    hq.hq_selftest_set_pipeline_stall(LIMIT, DELAY)
    try:
        call()
        status = hq.hq_read_device_error()
    finally:
        hq.hq_selftest_set_pipeline_stall(0, 0)
    assert status == hq.HQ_ERR_TIMEOUT, hq.hq_status_string(status)
    call()
    assert_no_device_error()
    check()
