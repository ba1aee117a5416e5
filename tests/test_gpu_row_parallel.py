"""The row-parallel layer in 8-bit integers against plain 64-bit arithmetic.

Codes, products and wires are compared for equality: a product's sum is an integer that doubles hold
exactly, and every later step is one rounded fp32 operation.  Norms are held to the roundings of
their steps: half a step of the stored type, and at most 128 fp32 roundings (a row's sum: up to 64
elements a thread, then 10 levels of a tree; the rest are a handful) of the terms' magnitudes.
"""
import pytest
import torch

import bit_tensor_activation_b200 as hq
from gpu_helpers import DEV, assert_no_device_error

pytestmark = pytest.mark.gpu
D = torch.float64
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _errors_are_clear():
    hq.hq_read_device_error()
    yield
    assert_no_device_error()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def pitched(t, pitch, fill=0):
    """`t` as a view of rows `pitch` elements apart, and the buffer behind it."""
    buf = torch.full((*t.shape[:-1], pitch), fill, dtype=t.dtype, device=t.device)
    buf[..., :t.shape[-1]] = t
    return buf[..., :t.shape[-1]], buf


def up(n, m):
    return -(-n // m) * m


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def same(got, want, what=""):
    got, want = got.contiguous(), want.contiguous()
    nan = torch.isnan(want) if want.is_floating_point() else torch.zeros_like(want, dtype=torch.bool)
    if want.is_floating_point():
        assert torch.equal(torch.isnan(got), nan), what
        got, want = bits(got), bits(want)
    bad = (got != want) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


# -------------------------------------------------------------------------------- tokens
def plain_tokens(x):
    """Codes and scales from the definition: the quotient in 64 bits (exactly tied or more than 2^-16 of
    itself off a tie, so that its own rounding does not matter)."""
    d = x.to(D)
    amax = d.abs().amax(-1, keepdim=True)
    scale = (amax / 127).float()  # in 64 bits: torch divides fp32 by a Python number through its reciprocal
    good = torch.isfinite(amax) & (scale >= torch.finfo(torch.float32).tiny)
    q = torch.where(good, torch.round(127 * d / torch.where(good, amax, 1)), 0)
    scale = torch.where(good, scale, torch.where(torch.isfinite(amax), 1.0, float("nan")))
    return torch.nan_to_num(q).to(torch.int8), scale[..., 0].float()


@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 8), (9, 255), (4, 256), (6, 257), (3, 512), (130, 1001),
                                    (33, 1024), (5, 1025), (7, 4097), (3, 8192), (2, 16392), (2, 32769), (2, 65536)])
def test_token_codes(rows, K):
    g = gen(rows * 100003 + K)
    x = (torch.randn(rows, K, generator=g, device=DEV) * torch.exp(3 * torch.randn(rows, 1, generator=g, device=DEV))).to(BF)
    x[0, K // 2] = x[0].abs().max() / 2  # an exact tie, 63.5
    xv, _ = pitched(x, up(K, 8) + 8, 7.0)
    q, buf = pitched(torch.full((rows, K), 99, dtype=torch.int8, device=DEV), up(K, 16) + 16, 99)
    s = torch.full((rows + 1,), -1.0, device=DEV)
    hq.hq_quantize_tokens(xv, q, s[:rows])
    want_q, want_s = plain_tokens(x)
    same(q, want_q, "codes")
    same(s[:rows], want_s, "scales")
    assert s[rows] == -1 and (buf[:, K:] == 99).all(), "written outside"


@pytest.mark.parametrize("K", [24, 700, 2000])
def test_token_rows_without_a_scale(K):
    nan, inf = float("nan"), float("inf")
    x = torch.ones(9, K, device=DEV)
    x[0], x[1, 3], x[2, K - 1], x[3, 0] = 0.0, nan, inf, -inf
    x[4] = 2.0 ** -126                     # amax / 127 subnormal
    x[5] = 127 * 2.0 ** -126               # amax / 127 the smallest normal number
    x[6] = -0.0
    x[7] = 3.3e38
    x[8] = 2.0 ** -133                     # subnormal bf16
    x = pitched(x.to(BF), up(K, 8))[0]
    q, s = torch.empty(9, up(K, 16), dtype=torch.int8, device=DEV)[:, :K], torch.empty(9, device=DEV)
    hq.hq_quantize_tokens(x, q, s)
    want_q, want_s = plain_tokens(x)
    same(q, want_q, "codes")
    same(s, want_s, "scales")
    assert (s[[0, 4, 6, 8]] == 1).all() and torch.isnan(s[1:4]).all() and (q[7] == 127).all()


def test_no_tokens():
    hq.hq_quantize_tokens(torch.empty(0, 16, dtype=BF, device=DEV), torch.empty(0, 16, dtype=torch.int8, device=DEV),
                          torch.empty(0, device=DEV))


# -------------------------------------------------------------------------------- products
def operands(seed, P, T, H, K, lda=0, ldw=0, full=False):
    g = gen(seed)
    lo = -128 if full else -127
    draw = lambda *s: torch.randint(lo, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    a, w = draw(P, T, K), draw(P, H, K)
    if full:
        a[..., :], w[..., :] = -128, -128
    av = pitched(a, lda or up(K, 16), 77)[0]
    wv = pitched(w, ldw or up(K, 16), 77)[0]
    a_s = torch.exp(torch.randn(P, T, generator=g, device=DEV)) / 127
    w_s = torch.exp(torch.randn(P, H, generator=g, device=DEV)) / 127
    return av, a_s, wv, w_s


def plain_product(a, a_s, w, w_s, bias=None):
    acc = torch.bmm(a.to(D), w.to(D).transpose(1, 2))  # integers below 2^31: exact
    v = acc.float() * a_s[..., None] * w_s[:, None]
    return v + bias.float()[:, None] if bias is not None else v


SHAPES = [  # P, T, H, K
    (1, 1, 8, 1), (1, 1, 64, 64), (2, 1, 4096, 512), (1, 2, 264, 100), (3, 5, 136, 129), (1, 16, 8192, 1024),
    (4, 32, 4096, 256), (2, 33, 520, 1001), (1, 64, 1000, 2048), (2, 65, 128, 128), (1, 100, 2056, 640),
    (3, 127, 256, 127), (2, 128, 256, 256), (1, 129, 264, 4096), (2, 200, 1032, 512), (1, 256, 512, 96),
    (8, 257, 248, 384), (1, 513, 4104, 65), (2, 1000, 1000, 1000), (64, 3, 24, 40), (1, 2, 40, 65536),
    (1, 300, 16, 20000), (2, 8, 48, 33000), (1, 24, 32776, 48), (1, 300, 65544, 16),
]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("P,T,H,K", SHAPES)
def test_product(P, T, H, K, f32):
    a, a_s, w, w_s = operands(P * 7 + T * 13 + H * 17 + K, P, T, H, K)
    bias = torch.randn(P, H, generator=gen(5), device=DEV).to(BF) if (T + K) % 2 else None
    t = torch.float32 if f32 else BF
    out = torch.full((P, T, H), 9.0, dtype=t, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, out, bias=bias)
    same(out, plain_product(a, a_s, w, w_s, bias).to(t), "out")


@pytest.mark.parametrize("P,T,H,K", [(2, 7, 72, 130), (1, 300, 520, 70), (3, 128, 256, 256), (1, 1, 264, 33)])
def test_product_of_wide_rows(P, T, H, K):
    """Rows further apart than their width on every side; nothing outside the block is written."""
    a, a_s, w, w_s = operands(3, P, T, H, K, lda=up(K, 16) + 48, ldw=up(K, 16) + 16)
    out, buf = pitched(torch.zeros(P, T, H, dtype=BF, device=DEV), H + 24, 5.0)
    hq.hq_int8_matmul(a, a_s, w, w_s, out)
    same(out, plain_product(a, a_s, w, w_s).to(BF), "out")
    assert (buf[..., H:] == 5).all()


@pytest.mark.parametrize("P,T,H,K", [(2, 9, 136, 200), (2, 300, 264, 272)])
def test_product_stays_in_its_rows(P, T, H, K):
    a, a_s, w, w_s = operands(4, P, T, H, K)
    for t in (BF, torch.float32):
        buf = torch.full((P * T * H + 4096,), 3.0, dtype=t, device=DEV)
        out = buf[2048:2048 + P * T * H].view(P, T, H)
        hq.hq_int8_matmul(a, a_s, w, w_s, out)
        same(out, plain_product(a, a_s, w, w_s).to(t), "out")
        assert (buf[:2048] == 3).all() and (buf[2048 + P * T * H:] == 3).all()


@pytest.mark.parametrize("T,K", [(1, 65536), (40, 65536), (200, 65536)])
def test_largest_sums(T, K):
    """Every operand -128: the sum is 2^30 at K = 65536."""
    a, a_s, w, w_s = operands(6, 1, T, 16, K, full=True)
    out = torch.empty(1, T, 16, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, out)
    same(out, plain_product(a, a_s, w, w_s), "out")
    assert torch.equal(out, (torch.full((), 2.0 ** 30, device=DEV) * a_s[..., None] * w_s[:, None]))


@pytest.mark.parametrize("T", [3, 200])
def test_scales_that_are_not_numbers_stay_in_their_rows(T):
    a, a_s, w, w_s = operands(8, 2, T, 264, 96)
    a_s[0, 1], a_s[1, 0], w_s[1, 7] = float("nan"), float("inf"), 0.0
    out = torch.empty(2, T, 264, dtype=BF, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, out)
    same(out, plain_product(a, a_s, w, w_s).to(BF), "out")
    assert torch.isnan(out[0, 1]).all() and not torch.isnan(out[0, 0]).any()
    assert (bits(out[0, 1]) == 0x7FC0).all()


def test_no_rows():
    a, a_s, w, w_s = operands(9, 2, 0, 64, 32)
    hq.hq_int8_matmul(a, a_s, w, w_s, torch.empty(2, 0, 64, dtype=BF, device=DEV))


def test_offsets_past_32_bits():
    """More than 2^32 output elements (8.6 GB) and an operand whose last rows lie past 2^31 bytes."""
    P, T, H, K = 2, 270_000, 8192, 16
    a, a_s, w, w_s = operands(10, P, T, H, K)
    out = torch.empty(P, T, H, dtype=BF, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, out)
    for r in range(P):
        for t0 in (0, 131_000, T - 300):
            sl = slice(t0, t0 + 300)
            same(out[r:r + 1, sl], plain_product(a[r:r + 1, sl], a_s[r:r + 1, sl], w[r:r + 1], w_s[r:r + 1]).to(BF), "out")
    del out
    a = torch.randint(-127, 128, (1, 36_000, 65_536), device=DEV, dtype=torch.int8)  # 2.4e9 bytes
    a_s = torch.rand(1, 36_000, device=DEV)
    w, w_s = torch.randint(-127, 128, (1, 64, 65_536), device=DEV, dtype=torch.int8), torch.rand(1, 64, device=DEV)
    out = torch.empty(1, 36_000, 64, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, out)
    for t0 in (0, 32_700, 35_872):
        same(out[:, t0:t0 + 128], plain_product(a[:, t0:t0 + 128], a_s[:, t0:t0 + 128], w, w_s), "out")


# -------------------------------------------------------------------------------- the wire
def selection(seed, P, H, k):
    g = gen(seed)
    perm = torch.randperm(H, generator=g, device=DEV)
    keep, rest = perm[:k].sort().values.int(), perm[k:].sort().values.int()
    zero = torch.randint(0, 16, (P, H), generator=g, device=DEV, dtype=torch.uint8)
    return keep, rest, zero


WIRE_SHAPES = [  # P, T, H, K, k
    (1, 1, 8, 5, 0), (1, 1, 8, 5, 8), (2, 3, 64, 40, 8), (4, 32, 4096, 256, 64), (1, 17, 1000, 129, 40),
    (3, 33, 264, 100, 264), (2, 40, 256, 96, 0), (2, 128, 256, 64, 8), (1, 129, 520, 200, 248), (8, 100, 2056, 65, 16),
    (2, 300, 4104, 512, 128), (1, 1, 32768, 64, 1024), (3, 257, 1032, 1001, 504),
]


@pytest.mark.parametrize("P,T,H,K,k", WIRE_SHAPES)
def test_wire_is_quantize_pack_of_the_product(P, T, H, K, k):
    a, a_s, w, w_s = operands(P + T + H + K + k, P, T, H, K)
    keep, rest, zero = selection(k + 1, P, H, k)
    x = torch.empty(P, T, H, dtype=BF, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, x)
    inv = (4 / x.float().std(1).clamp_min(1e-6) if T > 1 else 4 / x.float().abs().amax(1).clamp_min(1e-6)).contiguous()
    codes, side = torch.empty(P, T, (H - k) // 8, dtype=torch.int32, device=DEV), torch.empty(P, k, T, dtype=BF, device=DEV)
    hq.hq_quantize_pack(x, keep, rest, inv, zero, codes, side)
    order = torch.cat([rest, keep]).long()
    wo = pitched(w[:, order].contiguous(), up(K, 16))[0]
    pad = 64
    cbuf = torch.full((codes.numel() + 2 * pad,), 0x5A5A5A5A, dtype=torch.int32, device=DEV)
    sbuf = torch.full((side.numel() + 2 * pad,), 3.0, dtype=BF, device=DEV)
    got_c, got_s = cbuf[pad:pad + codes.numel()].view_as(codes), sbuf[pad:pad + side.numel()].view_as(side)
    hq.hq_int8_matmul_pack(a, a_s, wo, w_s[:, order].contiguous(), keep, rest, inv, zero, got_c, got_s)
    same(got_c, codes, "codes")
    same(got_s, side, "side")
    for b, v in ((cbuf, 0x5A5A5A5A), (sbuf, 3.0)):
        assert (b[:pad] == v).all() and (b[len(b) - pad:] == v).all(), "written outside"


@pytest.mark.parametrize("T", [4, 150])
def test_wire_of_values_that_are_not_numbers(T):
    """NaN takes the zero point's code, infinities and what is out of range saturate, as in quantize-pack."""
    P, H, K, k = 2, 272, 48, 16
    a, a_s, w, w_s = operands(12, P, T, H, K)
    keep, rest, zero = selection(3, P, H, k)
    a_s[0, 0], a_s[0, 1], a_s[1, 2] = float("nan"), float("inf"), 1e30
    inv = torch.full((P, H), 1e-3, device=DEV)
    inv[1, 5], inv[0, 9] = float("inf"), 0.0
    x = torch.empty(P, T, H, dtype=BF, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, x)
    want = torch.empty(P, T, (H - k) // 8, dtype=torch.int32, device=DEV), torch.empty(P, k, T, dtype=BF, device=DEV)
    hq.hq_quantize_pack(x, keep, rest, inv, zero, *want)
    order = torch.cat([rest, keep]).long()
    got = torch.empty_like(want[0]), torch.empty_like(want[1])
    hq.hq_int8_matmul_pack(a, a_s, w[:, order].contiguous(), w_s[:, order].contiguous(), keep, rest, inv, zero, *got)
    same(got[0], want[0], "codes")
    same(got[1], want[1], "side")


@pytest.mark.parametrize("T", [3, 200])
def test_a_bad_feature_index_is_reported(T):
    P, H, K, k = 1, 64, 32, 8
    a, a_s, w, w_s = operands(13, P, T, H, K)
    keep, rest, zero = selection(4, P, H, k)
    rest[3] = H + 5
    hq.hq_int8_matmul_pack(a, a_s, w, w_s, keep, rest, torch.ones(P, H, device=DEV), zero,
                           torch.empty(P, T, (H - k) // 8, dtype=torch.int32, device=DEV),
                           torch.empty(P, k, T, dtype=BF, device=DEV))
    assert hq.hq_read_device_error() == hq.HQ_ERR_BAD_INDEX


# -------------------------------------------------------------------------------- the block's end
STEPS = 128 * 2.0 ** -24


def plain_norm(x, kind, w, b, eps):
    """(norm, the magnitude its fp32 roundings are relative to), both in 64 bits."""
    x = x.to(D)
    if kind == hq.HQ_NORM_NONE:
        return x, torch.zeros_like(x)
    mag = x.abs()
    if kind == hq.HQ_NORM_LAYER:
        mag = mag + mag.mean(-1, keepdim=True)
        x = x - x.mean(-1, keepdim=True)
    var = x.square().mean(-1, keepdim=True)
    # of the centred values a mean off by d (relative d of the magnitude) moves the variance by 2 x d
    slack = (mag.square().mean(-1, keepdim=True) / var.clamp_min(1e-300)).sqrt()
    rstd = (var + eps).rsqrt()
    w = torch.ones(x.shape[-1], dtype=D, device=DEV) if w is None else w.to(D)
    b = torch.zeros(x.shape[-1], dtype=D, device=DEV) if b is None else b.to(D)
    n = x * rstd * w
    return n + b, (mag * rstd * w.abs() + n.abs() * slack) + b.abs()


def close(got, want, mag, what):
    half = torch.finfo(got.dtype).eps / 2
    off = (got.to(D) - want).abs() - half * want.abs() - STEPS * mag * (1 + half)
    assert (off <= torch.finfo(got.dtype).tiny).all(), f"{what}: over its bound by {float(off.max())}"


NORM_SHAPES = [(1, 8), (3, 16), (5, 256), (2, 264), (9, 520), (4, 1024), (7, 1032), (1, 4096), (32, 8192), (3, 5000),
               (2, 8200), (5, 16384), (2, 32768), (300, 2048), (6, 656), (5, 768), (4, 776)]


@pytest.mark.parametrize("kinds", [("none", "rms"), ("rms", "rms"), ("layer", "layer"), ("rms", "none"), ("layer", "rms")],
                         ids="-".join)
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_residual_norm(T, H, kinds):
    kind = {"none": hq.HQ_NORM_NONE, "rms": hq.HQ_NORM_RMS, "layer": hq.HQ_NORM_LAYER}
    post, pre = kind[kinds[0]], kind[kinds[1]]
    seed = T * 31 + H + post * 5 + pre
    g = gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    y_t, r_t = (BF, torch.float32)[seed & 1], (BF, torch.float32)[(seed >> 1) & 1]
    y, res = (2 * rnd(T, H) + 0.5).to(y_t), (rnd(T, H) * torch.exp(rnd(H))).to(r_t)
    y[0] = 0  # a row of zeros: its norm is zero (rms), or the bias
    post_w, post_b = (1 + rnd(H) / 4, rnd(H) / 4) if post else (None, None)
    pre_w, pre_b = (1 + rnd(H) / 4, rnd(H) / 4) if pre and seed % 3 else (None, None)
    G = [0, 1, T][seed % 3]
    gate = torch.tanh(rnd(G, H)).to(BF) if G else None
    alpha, beta, eps = 0.75, -1.25, 1e-5
    out = torch.empty(T, H, dtype=r_t, device=DEV)
    h = torch.empty(T, H, dtype=BF, device=DEV) if pre else None
    q, q_buf = pitched(torch.zeros(T, H, dtype=torch.int8, device=DEV), up(H, 16) + 16, 55) if pre else (None, None)
    q_s = torch.empty(T, device=DEV) if pre else None
    hq.hq_residual_norm(y, res, out, h=h, q=q, q_scale=q_s, post=post, post_w=post_w, post_b=post_b, gate=gate,
                        alpha=alpha, beta=beta, pre=pre, pre_w=pre_w, pre_b=pre_b, eps=eps)
    u, mag = plain_norm(y, post, post_w, post_b, eps)
    gt = gate.to(D).repeat_interleave(T // G, 0) if G else torch.ones(1, dtype=D, device=DEV)
    want = alpha * res.to(D) + beta * gt * u
    close(out, want, (alpha * res.to(D)).abs() + (beta * gt * u).abs() + (beta * gt).abs() * mag, "residual")
    if pre:
        n, mag = plain_norm(out, pre, pre_w, pre_b, eps)
        close(h, n, mag, "h")
        want_q, want_s = plain_tokens(h)
        same(q, want_q, "codes")
        same(q_s, want_s, "scales")
        assert (q_buf[:, H:] == 55).all()
        # the same without h, and with the residual in place
        q2, s2, res2 = torch.empty(T, up(H, 16), dtype=torch.int8, device=DEV)[:, :H], torch.empty(T, device=DEV), res.clone()
        hq.hq_residual_norm(y, res2, res2, q=q2, q_scale=s2, post=post, post_w=post_w, post_b=post_b, gate=gate,
                            alpha=alpha, beta=beta, pre=pre, pre_w=pre_w, pre_b=pre_b, eps=eps)
        same(res2, out, "in place")
        same(q2, q, "codes without h")
        same(s2, q_s, "scales without h")


def test_gate_rows_of_sequences():
    """Four sequences of three rows, each with its own gate; the first of them shut."""
    T, H = 12, 72
    y, res = torch.randn(T, H, device=DEV).to(BF), torch.randn(T, H, device=DEV).to(BF)
    gate = torch.randn(4, H, device=DEV).to(BF)
    gate[0] = 0
    out, h = torch.empty_like(res), torch.empty_like(res)
    hq.hq_residual_norm(y, res, out, h=h, gate=gate)
    want = res.to(D) + gate.to(D).repeat_interleave(3, 0) * y.to(D)
    close(out, want, want.abs() + res.to(D).abs(), "residual")
    same(out[:3], res[:3], "shut gate")


@pytest.mark.parametrize("H", [64, 4096])
def test_norm_rows_that_are_not_numbers(H):
    """A row with a NaN or an infinity is NaN throughout its norm and leaves the others alone."""
    y, res = torch.randn(6, H, device=DEV).to(BF), torch.randn(6, H, device=DEV).to(BF)
    y[1, 3], y[4, H - 1] = float("nan"), float("inf")
    out, h = torch.empty_like(res), torch.empty_like(res)
    q, s = torch.empty(6, H, dtype=torch.int8, device=DEV), torch.empty(6, device=DEV)
    hq.hq_residual_norm(y, res, out, h=h, q=q, q_scale=s, post=hq.HQ_NORM_RMS, pre=hq.HQ_NORM_RMS)
    bad = torch.tensor([False, True, False, False, True, False], device=DEV)
    assert torch.equal(torch.isnan(h).any(1), bad) and torch.equal(torch.isnan(s), bad)
    assert (q[bad] == 0).all() and torch.isfinite(h[~bad]).all()


def test_no_rows_to_norm():
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    hq.hq_residual_norm(e, e, e, h=e, gate=torch.empty(1, 64, dtype=BF, device=DEV))


# -------------------------------------------------------------------------------- together
def layer(x, w, w_s, sel, res, up_w, up_s, b, stream=None):
    keep, rest, scale, inv, zero = sel
    hq.hq_quantize_tokens(x, b["a"], b["a_s"], stream=stream)
    hq.hq_int8_matmul_pack(b["a"], b["a_s"], w, w_s, keep, rest, inv, zero, b["codes"], b["side"], stream=stream)
    hq.hq_dequant_reduce(b["codes"], b["side"], keep, rest, scale, zero, b["sum"], stream=stream)
    hq.hq_residual_norm(b["sum"], res, b["res"], q=b["q"], q_scale=b["q_s"], post=hq.HQ_NORM_RMS, stream=stream)
    hq.hq_int8_matmul(b["q"][None], b["q_s"][None], up_w, up_s, b["up"], stream=stream)


def layer_problem(seed, P, T, H, K, k, F):
    a, a_s, w, w_s = operands(seed, P, T, H, K)
    x = (a.float() * a_s[..., None]).to(BF).contiguous()
    keep, rest, zero = selection(seed, P, H, k)
    scale = torch.full((P, H), 0.25, device=DEV) * float(a_s.mean() * w_s.mean()) * 127 * 64 * K ** 0.5
    order = torch.cat([rest, keep]).long()
    up_w, up_s = torch.randint(-127, 128, (1, F, H), device=DEV, dtype=torch.int8), torch.rand(1, F, device=DEV)
    b = dict(a=torch.empty(P, T, up(K, 16), dtype=torch.int8, device=DEV)[..., :K], a_s=torch.empty(P, T, device=DEV),
             codes=torch.empty(P, T, (H - k) // 8, dtype=torch.int32, device=DEV),
             side=torch.empty(P, k, T, dtype=BF, device=DEV), sum=torch.empty(T, H, dtype=BF, device=DEV),
             res=torch.empty(T, H, dtype=BF, device=DEV), q=torch.empty(T, H, dtype=torch.int8, device=DEV),
             q_s=torch.empty(T, device=DEV), up=torch.empty(1, T, F, dtype=BF, device=DEV))
    res = torch.randn(T, H, generator=gen(seed), device=DEV).to(BF)
    return (x, w[:, order].contiguous(), w_s[:, order].contiguous(), (keep, rest, scale, (1 / scale).contiguous(), zero), res,
            up_w, up_s, b), (w, w_s)


def expected_layer(args, natural):
    """The same layer step by step: product, quantize-pack, reduction, norm in 64 bits, product."""
    x, _, _, (keep, rest, scale, inv, zero), res, up_w, up_s, b = args
    q, s = plain_tokens(x)
    part = plain_product(q, s, *natural).to(BF)
    P, T, H = part.shape
    codes, side = torch.empty_like(b["codes"]), torch.empty_like(b["side"])
    hq.hq_quantize_pack(part, keep, rest, inv, zero, codes, side)
    out = torch.empty(T, H, dtype=BF, device=DEV)
    hq.hq_dequant_reduce(codes, side, keep, rest, scale, zero, out)
    return out


@pytest.mark.parametrize("P,T,H,K,k,F", [(4, 32, 1024, 256, 64, 512), (2, 200, 528, 144, 16, 264), (1, 1, 256, 64, 0, 128)])
def test_a_layer_as_it_is_used(P, T, H, K, k, F):
    args, natural = layer_problem(21, P, T, H, K, k, F)
    b = args[-1]
    layer(*args)
    same(b["sum"], expected_layer(args, natural), "the ranks' sum")
    u, mag = plain_norm(b["sum"], hq.HQ_NORM_RMS, None, None, 1e-6)
    want = args[4].to(D) + u
    close(b["res"], want, want.abs() + mag, "residual")
    same(b["up"], plain_product(b["q"][None], b["q_s"][None], args[5], args[6]).to(BF), "next projection")


def test_captured_replayed_and_beside_another():
    """A captured layer replays on new inputs; two layers on two streams give what each gives alone."""
    args, natural = layer_problem(22, 2, 40, 1024, 512, 32, 256)
    other, other_natural = layer_problem(23, 3, 180, 528, 128, 16, 128)
    layer(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(*args)
    for seed in (1, 2):
        args[0].copy_(torch.randn(args[0].shape, generator=gen(seed), device=DEV).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        same(args[-1]["sum"], expected_layer(args, natural), "replay")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        layer(*args, stream=s1)
        layer(*other, stream=s2)
    torch.cuda.synchronize()
    same(args[-1]["sum"], expected_layer(args, natural), "first stream")
    same(other[-1]["sum"], expected_layer(other, other_natural), "second stream")


def test_one_product_as_two_captured_graphs_and_eagerly():
    """Two graphs of the same operands and an eager call, interleaved: no state is shared between them."""
    a, a_s, w, w_s = operands(31, 2, 8, 1024, 2048)
    outs = [torch.empty(2, 8, 1024, dtype=BF, device=DEV) for _ in range(3)]
    hq.hq_int8_matmul(a, a_s, w, w_s, outs[2])
    graphs = []
    for o in outs[:2]:
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            hq.hq_int8_matmul(a, a_s, w, w_s, o)
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        hq.hq_int8_matmul(a, a_s, w, w_s, outs[2])
    torch.cuda.synchronize()
    want = plain_product(a, a_s, w, w_s).to(BF)
    for o in outs:
        same(o, want, "out")


# -------------------------------------------------------------------------------- refusals of the binding
def test_refusals():
    a, a_s, w, w_s = operands(41, 2, 4, 64, 48)
    out = torch.full((2, 4, 64), 7.0, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        hq.hq_int8_matmul(a, a_s[:1], w, w_s, out)
    with pytest.raises(ValueError):
        hq.hq_int8_matmul(a.transpose(0, 1).contiguous().transpose(0, 1), a_s, w, w_s, out)  # ranks interleaved
    with pytest.raises(TypeError):
        hq.hq_int8_matmul(a.to(torch.uint8), a_s, w, w_s, out)
    with pytest.raises(TypeError):
        hq.hq_int8_matmul(a, a_s, w, w_s, out, bias=torch.zeros(2, 64, device=DEV))
    with pytest.raises(hq.HQError):
        hq.hq_int8_matmul(a[..., 8:], a_s, w[..., 8:], w_s, out)  # 8-byte aligned
    with pytest.raises(hq.HQError):
        hq.hq_int8_matmul(a[..., :40].contiguous(), a_s, w[..., :40].contiguous(), w_s, out)  # a pitch of 40
    x = torch.zeros(4, 12, dtype=BF, device=DEV)
    with pytest.raises(hq.HQError):
        hq.hq_quantize_tokens(x, torch.empty(4, 16, dtype=torch.int8, device=DEV)[:, :12], torch.empty(4, device=DEV))
    y = torch.zeros(4, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        hq.hq_residual_norm(y, y, out[0], h=y.clone(), gate=torch.zeros(3, 64, dtype=BF, device=DEV))
    with pytest.raises(TypeError):
        hq.hq_residual_norm(y, y.float(), out[0], h=y.clone())
    with pytest.raises(hq.HQError):
        hq.hq_residual_norm(y, y, out[0])
    torch.cuda.synchronize()
    assert (out == 7).all()


# -------------------------------------------------------------------------------- many rows to norm
@pytest.mark.parametrize("T,H,kinds,gates", [(1184, 8192, ("rms", "rms"), 1), (1300, 4104, ("layer", "layer"), 0),
                                             (1190, 5000, ("none", "rms"), 1190), (1200, 8192, ("rms", "none"), 3)])
@pytest.mark.parametrize("y_t,r_t", [(BF, BF), (torch.float32, BF), (BF, torch.float32), (torch.float32, torch.float32)],
                         ids=["bf16", "f32-bf16", "bf16-f32", "f32"])
def test_residual_norm_of_many_rows(T, H, kinds, gates, y_t, r_t):
    """Enough rows for the kernel that keeps weights in registers and rows in a ring."""
    kind = {"none": hq.HQ_NORM_NONE, "rms": hq.HQ_NORM_RMS, "layer": hq.HQ_NORM_LAYER}
    post, pre = kind[kinds[0]], kind[kinds[1]]
    g = gen(T + H)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    y, res = (2 * rnd(T, H) + 0.5).to(y_t), rnd(T, H).to(r_t)
    post_w, pre_w = 1 + rnd(H) / 4 if post else None, 1 + rnd(H) / 4 if pre else None
    gate = torch.tanh(rnd(gates, H)).to(BF) if gates else None
    buf = torch.full((T + 2, H), 7.0, dtype=r_t, device=DEV)
    out = buf[1:T + 1]
    h = torch.empty(T, H, dtype=BF, device=DEV) if pre else None
    q, q_s = (torch.empty(T, up(H, 16), dtype=torch.int8, device=DEV)[:, :H], torch.empty(T, device=DEV)) if pre else (None, None)
    hq.hq_residual_norm(y, res, out, h=h, q=q, q_scale=q_s, post=post, post_w=post_w, gate=gate, alpha=0.5, beta=2.0,
                        pre=pre, pre_w=pre_w, eps=1e-5)
    u, mag = plain_norm(y, post, post_w, None, 1e-5)
    gt = gate.to(D).repeat_interleave(T // gates, 0) if gates else torch.ones(1, dtype=D, device=DEV)
    want = 0.5 * res.to(D) + 2 * gt * u
    close(out, want, (0.5 * res.to(D)).abs() + (2 * gt * u).abs() + (2 * gt).abs() * mag, "residual")
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    if pre:
        n, mag = plain_norm(out, pre, pre_w, None, 1e-5)
        close(h, n, mag, "h")
        want_q, want_s = plain_tokens(h)
        same(q, want_q, "codes")
        same(q_s, want_s, "scales")
    res2 = res.clone()  # in place: rows are read ahead of their writing, never behind it
    hq.hq_residual_norm(y, res2, res2, h=h, post=post, post_w=post_w, gate=gate, alpha=0.5, beta=2.0, pre=pre, pre_w=pre_w,
                        eps=1e-5)
    same(res2, out, "in place")


# -------------------------------------------------------------------------------- one call after another
@pytest.mark.parametrize("T,H", [(1200, 5000), (300, 2056), (40, 520)])
def test_in_place_residuals_in_a_row(T, H):
    """Every call reads the residual that the call ahead wrote, in lines that two rows share: the same with
    nothing between the calls as with a wait after each."""
    y = torch.randn(8, T, H, generator=gen(T), device=DEV).to(BF)
    start = torch.randn(T, H, generator=gen(H), device=DEV).to(BF)
    got = []
    for wait in (True, False):
        res, h = start.clone(), torch.empty(T, H, dtype=BF, device=DEV)
        torch.cuda.synchronize()
        for i in range(40):
            hq.hq_residual_norm(h if i % 3 == 2 else y[i % 8], res, res, h=h if i % 3 != 2 else torch.empty_like(h),
                                post=hq.HQ_NORM_RMS, beta=0.5)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        got.append((res, h))
    same(got[1][0], got[0][0], "residual")
    same(got[1][1], got[0][1], "h")


@pytest.mark.parametrize("T", [3, 40, 200])
def test_operands_written_just_before_the_call(T):
    """Weights, scales and activations that the kernels just ahead in the stream are still writing."""
    P, H, K = 2, 1032, 200
    a, a_s, w, w_s = operands(51, P, T, H, K)
    xs = [(torch.randn(P, T, K, generator=gen(i), device=DEV) * (i + 1)).to(BF) for i in range(12)]
    x, q, s = torch.empty_like(xs[0]), torch.empty(P, T, 208, dtype=torch.int8, device=DEV)[..., :K], torch.empty(P, T, device=DEV)
    ww, ws = w.clone(), w_s.clone()
    outs = [torch.empty(P, T, H, dtype=torch.float32, device=DEV) for _ in xs]
    ww = pitched(w, up(K, 16))[0]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        x.copy_(xs[i])
        hq.hq_quantize_tokens(x, q, s)
        if i % 2:
            ww.neg_()
        else:
            ws.mul_(0.5)
        hq.hq_int8_matmul(q, s, ww, ws, o)
    torch.cuda.synchronize()
    sign, scale = 1, w_s.clone()
    for i, o in enumerate(outs):
        if i % 2:
            sign = -sign
        else:
            scale = scale * 0.5
        want_q, want_s = plain_tokens(xs[i])
        same(o, plain_product(want_q, want_s, sign * w, scale), f"call {i}")


@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_codes_that_start_anywhere(T, shift):
    """The codes need no more than 4-byte alignment, whatever their rows' length allows."""
    P, H, K, k = 2, 544, 96, 32
    a, a_s, w, w_s = operands(61, P, T, H, K)
    keep, rest, zero = selection(62, P, H, k)
    inv = torch.full((P, H), 1e-2, device=DEV)
    order = torch.cat([rest, keep]).long()
    wo, so = w[:, order].contiguous(), w_s[:, order].contiguous()
    n = P * T * (H - k) // 8
    want = torch.empty(P, T, (H - k) // 8, dtype=torch.int32, device=DEV), torch.empty(P, k, T, dtype=BF, device=DEV)
    hq.hq_quantize_pack(plain_product(a, a_s, w, w_s).to(BF), keep, rest, inv, zero, *want)
    buf = torch.full((n + 16,), 0x77, dtype=torch.int32, device=DEV)
    codes, side = buf[shift:shift + n].view_as(want[0]), torch.empty_like(want[1])
    hq.hq_int8_matmul_pack(a, a_s, wo, so, keep, rest, inv, zero, codes, side)
    same(codes, want[0], "codes")
    same(side, want[1], "side")
    assert (buf[:shift] == 0x77).all() and (buf[shift + n:] == 0x77).all()


@pytest.mark.parametrize("rows,K", [(1000, 9), (1001, 64), (999, 100), (1003, 128), (777, 250), (700, 256), (1201, 1500),
                                    (1200, 2048), (700, 2049), (640, 4097), (601, 8192), (600, 8193), (600, 20000)])
def test_token_codes_of_many_rows(rows, K):
    """Rows enough for every way in which a row's elements are shared, with rows over at the end."""
    g = gen(rows + K)
    x = (torch.randn(rows, K, generator=g, device=DEV) * torch.exp(2 * torch.randn(rows, 1, generator=g, device=DEV))).to(BF)
    x[rows // 2] = 0
    x[rows - 1, K - 1] = float("nan")
    xv, _ = pitched(x, up(K, 8) + 8, 7.0)
    q, buf = pitched(torch.full((rows + 1, K), 99, dtype=torch.int8, device=DEV), up(K, 16) + 16, 99)
    s = torch.full((rows + 1,), -1.0, device=DEV)
    hq.hq_quantize_tokens(xv, q[:rows], s[:rows])
    want_q, want_s = plain_tokens(x)
    same(q[:rows], want_q, "codes")
    same(s[:rows], want_s, "scales")
    assert s[rows] == -1 and (buf[:, K:] == 99).all() and (buf[rows] == 99).all(), "written outside"


# -------------------------------------------------------------------------------- what the documentation allows besides
def test_tokens_of_any_rank():
    """[..., K]: a single row without a leading dimension, and rows in three of them."""
    x = torch.randn(40, generator=gen(1), device=DEV).to(BF)
    q, s = torch.empty(48, dtype=torch.int8, device=DEV)[:40], torch.empty((), device=DEV)
    hq.hq_quantize_tokens(x, q, s)
    want_q, want_s = plain_tokens(x[None])
    same(q, want_q[0], "codes")
    same(s[None], want_s, "scale")
    x = torch.randn(2, 3, 5, 64, generator=gen(2), device=DEV).to(BF)
    q, s = torch.empty(2, 3, 5, 64, dtype=torch.int8, device=DEV), torch.empty(2, 3, 5, device=DEV)
    hq.hq_quantize_tokens(x, q, s)
    want_q, want_s = plain_tokens(x)
    same(q, want_q, "codes")
    same(s, want_s, "scales")
    with pytest.raises(ValueError):  # rows that are not one pitch apart
        hq.hq_quantize_tokens(x.transpose(0, 1), q.transpose(0, 1), torch.empty(3, 2, 5, device=DEV))


def test_no_rows_of_a_wire():
    a, a_s, w, w_s = operands(71, 2, 0, 64, 32)
    keep, rest, zero = selection(72, 2, 64, 8)
    hq.hq_int8_matmul_pack(a, a_s, w, w_s, keep, rest, torch.ones(2, 64, device=DEV), zero,
                           torch.empty(2, 0, 7, dtype=torch.int32, device=DEV), torch.empty(2, 8, 0, dtype=BF, device=DEV))


@pytest.mark.parametrize("T,H,rows", [(10, 64, 4), (1301, 8192, 100), (500, 4096, 499)])
def test_gate_rows_that_do_not_divide_the_tokens(T, H, rows):
    """The C call's gate has ceil(T / gate_rows) rows, the last of them for what is left."""
    G = -(-T // rows)
    y, res, gate = (torch.randn(n, H, generator=gen(n + H), device=DEV).to(BF) for n in (T, T + 1, G))
    res = res[:T]
    out, h = torch.empty(T, H, dtype=BF, device=DEV), torch.empty(T, H, dtype=BF, device=DEV)
    torch.cuda.synchronize()
    st = hq.lib().hq_residual_norm(y.data_ptr(), 0, res.data_ptr(), out.data_ptr(), 0, T, H, 0, None, None, gate.data_ptr(),
                                   rows, 1.0, 1.0, 1, None, None, 1e-6, h.data_ptr(), None, 0, None, None)
    assert st == hq.HQ_OK
    torch.cuda.synchronize()
    u = gate.to(D)[torch.arange(T, device=DEV) // rows] * y.to(D)
    close(out, res.to(D) + u, res.to(D).abs() + u.abs(), "residual")


def test_bits_and_parameters_as_tensors():
    """bf16 tensors may be passed as their bits, and weights as parameters that ask for gradients."""
    a, a_s, w, w_s = operands(81, 1, 5, 64, 48)
    out = torch.empty(1, 5, 64, dtype=torch.int16, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, torch.nn.Parameter(w_s), out)
    same(out.view(BF), plain_product(a, a_s, w, w_s).to(BF), "out")


def test_many_features():
    """The largest number of features of a product."""
    P, T, H, K = 1, 3, hq.HQ_INT8_MAX_H, 32
    a, a_s, w, w_s = operands(91, P, T, H, K)
    out = torch.empty(P, T, H, dtype=BF, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, out)
    same(out, plain_product(a, a_s, w, w_s).to(BF), "few tokens")
    T = 70
    a, a_s, w, w_s = operands(92, P, T, H, K)
    out = torch.empty(P, T, H, dtype=BF, device=DEV)
    hq.hq_int8_matmul(a, a_s, w, w_s, out)
    same(out, plain_product(a, a_s, w, w_s).to(BF), "more tokens")
