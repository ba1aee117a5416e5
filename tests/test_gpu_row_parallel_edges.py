"""Where the row-parallel layer's kernels and calls can go wrong besides their sizes: lanes of a warp that
part ways, waits that run out at any moment, sizes past 32 bits, arguments of every kind.

Plain forms and tolerances are those of test_gpu_row_parallel.py: codes, products and wires are compared
for equality.
"""
import pytest
import torch

import bit_tensor_activation_b200 as hq
from gpu_helpers import DEV, assert_no_device_error
from test_gpu_row_parallel import BF, expected_layer, layer, layer_problem, operands, plain_product, plain_tokens, same, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _errors_are_clear():
    hq.hq_read_device_error()
    yield
    assert_no_device_error()


def wire_problem(seed, P, T, H, K, k, inv=1e-2):
    """A product's operands, the wire's parameters and the weights in the wire's order."""
    a, a_s, w, w_s = operands(seed, P, T, H, K)
    keep, rest, zero = selection(seed, P, H, k)
    order = torch.cat([rest, keep]).long()
    wo = torch.zeros(P, H, -(-K // 16) * 16, dtype=torch.int8, device=DEV)
    wo[..., :K] = w[:, order]
    return a, a_s, w, w_s, wo[..., :K], w_s[:, order].contiguous(), keep, rest, torch.full((P, H), inv, device=DEV), zero


def empty_wire(P, T, H, k):
    return (torch.empty(P, T, (H - k) // 8, dtype=torch.int32, device=DEV), torch.empty(P, k, T, dtype=BF, device=DEV))


def check_wire(problem, k):
    a, a_s, w, w_s, wo, so, keep, rest, inv, zero = problem
    P, T, H = a.shape[0], a.shape[1], w.shape[1]
    want, got = empty_wire(P, T, H, k), empty_wire(P, T, H, k)
    hq.hq_quantize_pack(plain_product(a, a_s, w, w_s).to(BF), keep, rest, inv, zero, *want)
    hq.hq_int8_matmul_pack(a, a_s, wo, so, keep, rest, inv, zero, *got)
    same(got[0], want[0], "codes")
    same(got[1], want[1], "side")


# -------------------------------------------------------------------------------- lanes that part ways
@pytest.mark.parametrize("P,T,H,K,k", [(2, 300, 1056, 200, 40), (3, 70, 528, 96, 16), (1, 1001, 4096, 256, 64),
                                       (2, 33, 1032, 300, 264), (1, 64, 256, 1100, 8), (1, 5, 512, 4100, 16)])
def test_single_lanes_take_the_rare_path(P, T, H, K, k):
    """Every third token has a huge scale, every seventh is not a number, and kept features and the last
    tokens end within a warp: neighbouring lanes take different paths through one chunk after another."""
    problem = wire_problem(T + H, P, T, H, K, k)
    problem[1][:, ::3] *= 1e6
    problem[1][:, ::7] = float("nan")
    for _ in range(20):
        check_wire(problem, k)


@pytest.mark.parametrize("P,T,H,K", [(1, 1, 128, 4096), (1, 3, 264, 2048), (2, 16, 1000, 1024), (1, 20, 520, 1500),
                                     (1, 33, 4096, 8192), (1, 64, 1032, 4096), (1, 9, 512, 65536)])
def test_clusters_of_every_size(P, T, H, K):
    """K over two, four and eight CTAs, whose load and product warps come to the cluster's barrier from one
    lane's loop; the last features and tokens end within a warp."""
    a, a_s, w, w_s = operands(T + K, P, T, H, K)
    bias = torch.randn(P, H, device=DEV).to(BF)
    for t in (BF, torch.float32):
        want = plain_product(a, a_s, w, w_s, bias).to(t)
        for _ in range(20):
            out = torch.full((P, T, H), 9.0, dtype=t, device=DEV)
            hq.hq_int8_matmul(a, a_s, w, w_s, out, bias=bias)
            same(out, want, "out")


# -------------------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("what", ["few, its steps within the ring", "few", "few of a cluster", "pair, one tile", "pair",
                                  "pair, a tile's steps within the ring", "pair wire"])
def test_waits_that_run_out_at_any_moment(what):
    """Producers held back by 1 us to 0.5 ms, consumers that give up after about 0.2 ms: in some launches the
    wait runs out ahead of the loads, in some beside them, in some after the last of them was issued or in one
    CTA of several alone.  A launch either gives the result or reports HQ_ERR_TIMEOUT, with nothing of it under
    way when its CTAs leave, and the next one is right."""
    P, T, H, K = {"few, its steps within the ring": (2, 5, 8192, 300), "few": (8, 20, 8192, 3000),
                  "few of a cluster": (1, 9, 512, 4096), "pair, one tile": (1, 256, 256, 5000), "pair": (2, 600, 4096, 1500),
                  "pair, a tile's steps within the ring": (1, 100, 512, 600), "pair wire": (1, 700, 2048, 256)}[what]
    wire, k = what.endswith("wire"), 8
    problem = wire_problem(3, P, T, H, K, k)
    a, a_s, w, w_s, wo, so, keep, rest, inv, zero = problem
    want = plain_product(a, a_s, w, w_s).to(BF)
    if wire:
        codes, side = empty_wire(P, T, H, k)
        hq.hq_quantize_pack(want, keep, rest, inv, zero, codes, side)
        got = empty_wire(P, T, H, k)
    else:
        out = torch.empty(P, T, H, dtype=BF, device=DEV)

    def call():
        if wire:
            hq.hq_int8_matmul_pack(a, a_s, wo, so, keep, rest, inv, zero, *got)
        else:
            hq.hq_int8_matmul(a, a_s, w, w_s, out)

    def check():
        if wire:
            same(got[0], codes, "codes")
            same(got[1], side, "side")
        else:
            same(out, want, "out")

    assert_no_device_error()
    seen = []
    for delay in [2_000] + list(range(100_000, 500_000, 10_000)) + [1_000_000]:
        hq.hq_selftest_set_pipeline_stall(20_000, delay)
        try:
            call()
            seen.append(hq.hq_read_device_error())
        finally:
            hq.hq_selftest_set_pipeline_stall(0, 0)
        assert seen[-1] in (hq.HQ_OK, hq.HQ_ERR_TIMEOUT), hq.hq_status_string(seen[-1])
        if seen[-1] == hq.HQ_OK:
            check()
        call()
        assert_no_device_error()
        check()
    assert seen[-1] == hq.HQ_ERR_TIMEOUT


# -------------------------------------------------------------------------------- sizes at the limits of an int
def test_the_most_tokens():
    """T = 2^31 - 1, the largest that the call takes, as the narrowest wire (52 GB in all)."""
    P, T, H, K = 1, 2 ** 31 - 1, 8, 16
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of free memory")
    a = torch.zeros(P, T, K, dtype=torch.int8, device=DEV)
    a_s = torch.ones(P, T, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randint(-127, 128, (P, H, K), generator=g, device=DEV, dtype=torch.int8)
    w_s = torch.ones(P, H, device=DEV)
    ends = (slice(0, 300), slice(2 ** 30 - 150, 2 ** 30 + 150), slice(T - 300, T))
    for e in ends:
        a[:, e] = torch.randint(-127, 128, (P, 300, K), generator=g, device=DEV, dtype=torch.int8)
    keep, rest = torch.empty(0, dtype=torch.int32, device=DEV), torch.arange(H, dtype=torch.int32, device=DEV)
    inv = torch.full((P, H), 1e-4, device=DEV)
    zero = torch.arange(1, 9, dtype=torch.uint8, device=DEV).repeat(P, 2)[:, :H].contiguous()
    codes, side = torch.full((P, T, 1), 0x5A5A5A5A, dtype=torch.int32, device=DEV), torch.empty(P, 0, T, dtype=BF, device=DEV)
    hq.hq_int8_matmul_pack(a, a_s, w, w_s, keep, rest, inv, zero, codes, side)
    for e in ends:
        want = empty_wire(P, 300, H, 0)
        hq.hq_quantize_pack(plain_product(a[:, e], a_s[:, e], w, w_s).to(BF), keep, rest, inv, zero, *want)
        same(codes[:, e], want[0], "codes")
        assert len(want[0].unique()) > 100
        codes[:, e] = 0x87654321 - (1 << 32)  # the code of a row of zeros: the zero points
    for at in range(0, T, 1 << 28):
        assert (codes[:, at:at + (1 << 28)] == 0x87654321 - (1 << 32)).all()
    del a, a_s, codes
    torch.cuda.empty_cache()

# -------------------------------------------------------------------------------- indices out of range
@pytest.mark.parametrize("bad", [-1, 1 << 20, "H"])
@pytest.mark.parametrize("T", [3, 40, 200])
@pytest.mark.parametrize("kept,at", [(True, 0), (True, 23), (False, 0), (False, 500)])
def test_an_index_out_of_range_is_reported(T, kept, at, bad):
    """Of a kept feature as of another one."""
    P, H, K, k = 2, 1056, 48, 24
    _, _, _, _, wo, so, keep, rest, inv, zero = problem = wire_problem(5, P, T, H, K, k)
    codes, side = empty_wire(P, T, H, k)
    call = lambda: hq.hq_int8_matmul_pack(problem[0], problem[1], wo, so, keep, rest, inv, zero, codes, side)  # noqa: E731
    call()
    assert_no_device_error()
    (keep if kept else rest)[at] = H if bad == "H" else bad
    call()
    assert hq.hq_read_device_error() == hq.HQ_ERR_BAD_INDEX


# -------------------------------------------------------------------------------- again and again
@pytest.mark.parametrize("P,T,H,K,k,F", [(7, 1200, 280, 208, 0, 64), (3, 20, 1112, 272, 56, 616), (2, 700, 4104, 128, 40, 128)])
def test_a_layer_repeats_itself_bit_for_bit(P, T, H, K, k, F):
    """The same inputs give the same bits in every pass, alone and between passes on other inputs."""
    pairs = [list(layer_problem(seed, P, T, H, K, k, F)[0]) for seed in (31, 32)]
    for args in pairs:  # the product after the norm takes rows a multiple of 16 bytes apart
        args[-1]["q"] = torch.empty(T, -(-H // 16) * 16, dtype=torch.int8, device=DEV)[:, :H]
        rows = torch.zeros(*args[5].shape[:2], -(-H // 16) * 16, dtype=torch.int8, device=DEV)
        rows[..., :H] = args[5]
        args[5] = rows[..., :H]
    results = ("sum", "res", "q_s", "up", "codes")
    first = []
    for args in pairs:
        layer(*args)
        torch.cuda.synchronize()
        first.append({n: args[-1][n].clone() for n in results})
    for i in range(30):
        for args, want in zip(pairs, first):
            layer(*args)
            if i % 3 == 0:
                layer(*args)
            for n in results:
                same(args[-1][n], want[n], n)


# -------------------------------------------------------------------------------- other threads of the program
LOCK_SHIM = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stdio.h>
static int note(const char* name) {
  int (*held)(void) = (int (*)(void))dlsym(RTLD_DEFAULT, "PyGILState_Check");
  printf("%s %s\n", name, held && held() ? "held" : "free");
  fflush(stdout);
  return 0;
}
#define CALL(name) int name(void) { return note(#name); }
CALL(hq_quantize_tokens)
CALL(hq_int8_matmul)
CALL(hq_int8_matmul_pack)
CALL(hq_dequant_reduce)
CALL(hq_residual_norm)
"""
LOCK_PROGRAM = r"""
import torch
import bit_tensor_activation_b200 as hq
new = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
P, T, H, K, k = 2, 4, 64, 32, 8
i8, i32, u8, f32 = torch.int8, torch.int32, torch.uint8, torch.float32
a, a_s, w, w_s = new(P, T, K, dtype=i8), new(P, T, dtype=f32), new(P, H, K, dtype=i8), new(P, H, dtype=f32)
keep, rest, grid, zero = new(k, dtype=i32), new(H - k, dtype=i32), new(P, H, dtype=f32), new(P, H, dtype=u8)
codes, side, out = new(P, T, (H - k) // 8, dtype=i32), new(P, k, T), new(T, H)
hq.hq_quantize_tokens(new(P, T, K), a, a_s)
hq.hq_int8_matmul(a, a_s, w, w_s, new(P, T, H))
hq.hq_int8_matmul_pack(a, a_s, w, w_s, keep, rest, grid, zero, codes, side)
hq.hq_dequant_reduce(codes, side, keep, rest, grid, zero, out)
hq.hq_residual_norm(out, out, out, h=new(T, H))
"""


def test_launches_leave_pythons_lock_to_other_threads(tmp_path):
    """The library's calls are replaced by ones that launch nothing and say whether Python's lock is held."""
    import os
    import shutil
    import subprocess
    import sys

    if not shutil.which("gcc"):
        pytest.skip("needs a C compiler")
    (tmp_path / "shim.c").write_text(LOCK_SHIM)
    shim = str(tmp_path / "shim.so")
    subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / "shim.c"), "-o", shim, "-ldl"], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(hq.__file__)))
    r = subprocess.run([sys.executable, "-c", LOCK_PROGRAM], cwd=root, env=dict(os.environ, LD_PRELOAD=shim), text=True,
                       capture_output=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    said = dict(line.split() for line in r.stdout.splitlines() if line.startswith("hq_"))
    assert said == {n: "free" for n in ("hq_quantize_tokens", "hq_int8_matmul", "hq_int8_matmul_pack", "hq_dequant_reduce",
                                        "hq_residual_norm")}, said


# -------------------------------------------------------------------------------- both sets of argument checks
def calls_and_arguments():
    """Each call that C++ and Python both check, with arguments that fit."""
    new = lambda *s, dtype=BF: torch.ones(*s, dtype=dtype, device=DEV)  # noqa: E731
    P, T, H, K, k = 2, 4, 64, 48, 16
    i8, i32, u8, f32 = torch.int8, torch.int32, torch.uint8, torch.float32
    product = dict(a=new(P, T, K, dtype=i8), a_scale=new(P, T, dtype=f32), w=new(P, H, K, dtype=i8), w_scale=new(P, H, dtype=f32))
    wire = dict(keep_idx=torch.arange(k, dtype=i32, device=DEV), rest_idx=torch.arange(k, H, dtype=i32, device=DEV),
                codes=new(P, T, (H - k) // 8, dtype=i32), side=new(P, k, T), zero=new(P, H, dtype=u8))
    return {
        "quantize_tokens": dict(x=new(T, K), q=new(T, K, dtype=i8), scale=new(T, dtype=f32), stream=None),
        "int8_matmul": dict(**product, out=new(P, T, H), bias=new(P, H), stream=None),
        "int8_matmul_pack": dict(**product, keep_idx=wire["keep_idx"], rest_idx=wire["rest_idx"], inv_scale=new(P, H, dtype=f32),
                                 zero=wire["zero"], codes=wire["codes"], side=wire["side"], stream=None),
        "dequant_reduce": dict(codes=wire["codes"], side=wire["side"], keep_idx=wire["keep_idx"], rest_idx=wire["rest_idx"],
                               scale=new(P, H, dtype=f32), zero=wire["zero"], out=new(T, H), stream=None),
        "residual_norm": dict(y=new(T, H), res=new(T, H), res_out=new(T, H), h=new(T, H), q=new(T, H, dtype=i8),
                              q_scale=new(T, dtype=f32), post=1, post_w=new(H, dtype=f32), post_b=new(H, dtype=f32), gate=new(2, H),
                              alpha=1.0, beta=1.0, pre=2, pre_w=new(H, dtype=f32), pre_b=new(H, dtype=f32), eps=1e-6, stream=None),
    }


def variants(n, v):
    """Other values for argument `n`, most of which do not fit."""
    if n == "stream":  # a number is taken for a stream's handle: only numbers that are one
        yield from (("0", 0), ("a word", "x"), ("a stream", torch.cuda.current_stream(DEV)))
        return
    yield "None", None
    yield "a number", 3
    yield "a word", "x"
    if not isinstance(v, torch.Tensor):
        for x in (0, -1, 2, 5, 1.0, 0.5, True, 1e300, float("nan"), 2 ** 32 + 1, 10 ** 400, torch.tensor(1.0)):
            yield repr(x)[:20], x
        return
    wide = torch.empty(*v.shape[:-1], v.shape[-1] + 16, dtype=v.dtype, device=DEV).copy_(
        torch.nn.functional.pad(v.float(), (0, 16)).to(v.dtype))
    odd = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)[1:].view(v.shape).copy_(v)
    yield "on the host", v.cpu()
    yield "of another type", v.to(torch.float64)
    yield "fp32", v.float()
    yield "bf16", v.to(BF)
    yield "int32", v.to(torch.int32)
    if v.element_size() == 2:
        yield "bits", v.view(torch.int16)
        yield "unsigned bits", v.view(torch.uint16)
    if v.dtype == torch.int32:
        yield "unsigned", v.view(torch.uint32)
    yield "a dimension more", v[None]
    yield "a dimension less", v[0]
    yield "none of it", v[:0]
    yield "one of it", v[:1]
    yield "one less", v[:-1]
    yield "narrower", v[..., :-8]
    yield "with a pitch", wide[..., :v.shape[-1]]
    if v.dim() > 1:  # (shifted lists of features are not lists of features)
        yield "eight further", wide[..., 8:8 + v.shape[-1]]
    yield "misaligned", odd
    yield "every second", torch.cat([v, v], -1)[..., ::2]
    yield "repeated", v[:1].expand_as(v)
    if v.is_floating_point():
        yield "a parameter", torch.nn.Parameter(v)
    if v.dim() > 1:
        yield "transposed", v.transpose(0, 1)
        yield "columns first", v.transpose(-1, -2).contiguous().transpose(-1, -2)
    if v.dim() > 2:
        yield "ranks interleaved", v.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("name", ["quantize_tokens", "int8_matmul", "int8_matmul_pack", "dequant_reduce", "residual_norm"])
def test_both_checks_take_and_refuse_the_same(name, monkeypatch):
    """Every argument in turn in every other shape, type and place, and each pair of arguments cut to no rows:
    what the checks in C++ call the library with, those in Python do, and the library says the same of it."""
    public, fast = getattr(hq, "hq_" + name), getattr(hq._hqargs, name)

    class Slow:
        pass

    for n in ("quantize_tokens", "int8_matmul", "int8_matmul_pack", "dequant_reduce", "residual_norm"):
        setattr(Slow, n, staticmethod(lambda *args: None))
    monkeypatch.setattr(hq, "_hqargs", Slow)
    args = calls_and_arguments()[name]
    order = {"int8_matmul": ["a", "a_scale", "w", "w_scale", "out", "bias", "stream"]}.get(name, list(args))

    def both(kw, what):
        status = fast(*(hq._handle(kw[n]) if n == "stream" else kw[n] for n in order))
        try:
            public(**kw)
            other = hq.HQ_OK
        except hq.HQError as e:
            other = e.status
        except Exception:
            other = None
        assert status == other or (status is None and other), f"{name}, {what}: {status} in C++, {other} in Python"
        return status

    assert both(args, "as it is") == hq.HQ_OK
    seen = {both({**args, n: x}, f"{n} {what}") for n, v in args.items() for what, x in variants(n, v)}
    assert seen >= {None, hq.HQ_OK}
    tensors = [n for n, v in args.items() if isinstance(v, torch.Tensor)]
    for a in tensors:
        for b in tensors:
            both({**args, a: args[a][:0], b: args[b][:0]}, f"{a} and {b} of no rows")
            both({**args, a: None, b: None}, f"neither {a} nor {b}")
    empty = {n: v[:, :0] if v.dim() > 1 and v.shape[:2] == (2, 4) else v[..., :0] if n == "side" else
             v[:0] if v.shape[0] == 4 else v for n, v in args.items() if isinstance(v, torch.Tensor)}
    assert both({**args, **empty}, "no rows at all") == hq.HQ_OK
    torch.cuda.synchronize()


# -------------------------------------------------------------------------------- behind other streams and other work
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("T", [5, 50, 300])
def test_operands_from_another_stream(T, captured):
    """Weights and scales come from a slow stream that is joined just ahead of the product, the activations
    from a copy and a fill ahead of the quantizer; the norm behind reads a residual of that stream too."""
    P, H, K = 1, 528, 256
    side = torch.cuda.Stream()
    w, w_s = torch.zeros(P, H, K, dtype=torch.int8, device=DEV), torch.zeros(P, H, device=DEV)
    new_w, new_s = torch.empty_like(w), torch.empty_like(w_s)
    x, src = torch.zeros(P, T, K, dtype=BF, device=DEV), torch.empty(P, T, K, dtype=BF, device=DEV)
    q, s = torch.empty(P, T, K, dtype=torch.int8, device=DEV), torch.empty(P, T, device=DEV)
    out, res, new_res = torch.empty(P, T, H, dtype=BF, device=DEV), torch.zeros(T, H, dtype=BF, device=DEV), torch.empty(T, H, dtype=BF, device=DEV)
    h, r_out = torch.empty(T, H, dtype=BF, device=DEV), torch.empty(T, H, dtype=BF, device=DEV)
    slow = torch.randn(3000, 3000, device=DEV)
    sink = torch.empty_like(slow)

    def work():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(2):
                torch.mm(slow, slow, out=sink)
            w.copy_(new_w)
            w_s.copy_(new_s)
            ready = torch.cuda.Event()
            ready.record(side)
            torch.mm(slow, slow, out=sink)
            res.copy_(new_res)
        x.copy_(src)
        s.zero_()
        hq.hq_quantize_tokens(x, q, s)
        main.wait_event(ready)
        hq.hq_int8_matmul(q, s, w, w_s, out)
        main.wait_stream(side)
        hq.hq_residual_norm(out[0], res, r_out, h=h, post=hq.HQ_NORM_NONE)
        w.zero_()
        w_s.zero_()
        res.zero_()

    run = work
    if captured:
        work()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work()
        run = graph.replay
    for i in range(25):
        g = torch.Generator(device=DEV).manual_seed(i)
        src.copy_(torch.randn(P, T, K, generator=g, device=DEV).to(BF))
        new_w.copy_(torch.randint(-127, 128, (P, H, K), generator=g, device=DEV, dtype=torch.int8))
        new_s.copy_(torch.rand(P, H, generator=g, device=DEV) / 4096)
        new_res.copy_(torch.randn(T, H, generator=g, device=DEV).to(BF))
        torch.cuda.synchronize()
        run()
        if i % 2:
            run()
        torch.cuda.synchronize()
        codes, scales = plain_tokens(src)
        same(q, codes, "codes")
        want = plain_product(codes, scales, new_w, new_s).to(BF)
        same(out, want, "out")
        same(r_out, (new_res.float() + want[0].float()).to(BF), "residual")


def test_calls_through_the_checks_in_python(monkeypatch):
    """A layer, and a norm and a product with every optional argument, give the same bits without the C++ module."""
    args = layer_problem(41, 3, 40, 528, 144, 16, 264)[0]
    y, res, w, b = args[4], args[4].float(), torch.rand(528, device=DEV), torch.rand(528, device=DEV)
    gate, bias = torch.randn(4, 528, device=DEV).to(BF), torch.randn(3, 528, device=DEV).to(BF)
    a, a_s, ww, ws = operands(42, 3, 40, 528, 144)
    results = []
    for slow in (False, True):
        if slow:
            monkeypatch.setattr(hq, "_hqargs", hq._NoArgs)
        for n in ("sum", "res", "q", "q_s", "up", "codes", "side"):
            args[-1][n].fill_(3)
        layer(*args)
        out, h = torch.empty_like(res), torch.empty_like(y)
        q, q_s = torch.empty(40, 528, dtype=torch.int8, device=DEV), torch.empty(40, device=DEV)
        hq.hq_residual_norm(y, res, out, h=h, q=q, q_scale=q_s, post=hq.HQ_NORM_LAYER, post_w=w, post_b=b, gate=gate, alpha=0.5,
                            beta=2.0, pre=hq.HQ_NORM_RMS, pre_w=b, pre_b=w, eps=1e-3)
        part = torch.empty(3, 40, 528, device=DEV)
        hq.hq_int8_matmul(a, a_s, ww, ws, part, bias=bias)
        torch.cuda.synchronize()
        results.append([args[-1][n].clone() for n in ("sum", "res", "q", "q_s", "up", "codes", "side")] + [out, h, q, q_s, part])
    for i, (x, z) in enumerate(zip(*results)):
        same(z, x, f"output {i}")


def test_threads_that_call_at_once():
    """Four threads, each with a stream and a problem of its own, that reach several kernels for the first time
    together."""
    import threading

    problems = [layer_problem(50 + i, *sizes) for i, sizes in enumerate(
        [(2, 40, 1040, 256, 32, 136), (3, 130, 528, 144, 16, 264), (1, 7, 2064, 320, 0, 72), (2, 300, 272, 64, 16, 520)])]
    torch.cuda.synchronize()
    failed = []

    def work(args):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    layer(*args)
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(p[0],)) for p in problems]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for args, natural in problems:
        same(args[-1]["sum"], expected_layer(args, natural), "the ranks' sum")
        same(args[-1]["up"], plain_product(args[-1]["q"][None], args[-1]["q_s"][None], args[5], args[6]).to(BF), "next projection")
