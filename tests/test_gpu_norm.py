"""GPU parity of ida_rmsnorm and ida_rmsnorm_backward against the fp64 oracle (oracle/ida_ssm.py).

Bounds, from the arithmetic: half a step of the output's type on the value, plus 2^-24 times 64
(the roundings of a row's sum, at most 32 in a thread and 9 across threads, and of the products
behind it) on the terms it is made of; e4m3 values half a step (2^-4 of the value, 2^-10 of the
scale near zero).
"""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from oracle import ida_ssm as orc
from tests import ssm_cases as sc
from tests.ssm_cases import HALF, U32, worst

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _done():
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0


# (rows, D, dtype, residual, group)
NORMS = [(1, 8, "bf16", True, 0), (3, 8, "f32", False, 8), (5, 2048, "bf16", True, 0), (7, 768, "bf16", True, 128),
         (300, 2048, "bf16", True, 128), (33, 8192, "f32", True, 64), (9, 8192, "bf16", False, 8192),
         (2, 1000, "bf16", True, 1000), (17, 96, "f32", True, 32), (130, 1000, "f32", False, 0),
         (4000, 64, "bf16", True, 32), (2000, 4096, "bf16", True, 64), (11, 128, "bf16", True, 128),
         (1, 5000, "bf16", False, 0), (5000, 40, "f32", True, 40)]


def _inputs(rows, D, dtype, residual, seed=1):
    g = sc.gen(seed)
    x = (torch.randn(rows, D, generator=g) * 3).to(sc.DT[dtype])
    r = torch.randn(rows, D, generator=g).to(sc.DT[dtype]) if residual else None
    return x, r, 1 + 0.2 * torch.randn(D, generator=g)


@pytest.mark.parametrize("case", NORMS, ids=str)
def test_norm(case):
    rows, D, dtype, residual, group = case
    x, res, w = _inputs(rows, D, dtype, residual)
    want = torch.empty(rows, D, dtype=sc.DT[dtype], device="cuda")
    out, r, q, scale = binding.ida_rmsnorm(x.cuda(), w.cuda(), residual=None if res is None else res.cuda(), eps=EPS,
                                           group=group, out=want)
    _done()
    total = x.float() if res is None else x.float() + res.float()
    stored = total.to(sc.DT[dtype])
    assert torch.equal(r.cpu(), stored)
    y = orc.rmsnorm(stored.double(), w.double(), EPS)
    assert worst(out, y, (HALF[dtype] + 64 * U32) * y.abs()) <= 1
    if not group:
        assert q is None and scale is None
        return
    top = y.reshape(rows, -1, group).abs().amax(-1)
    assert worst(scale, top / 448, 64 * U32 * top / 448) <= 1
    s = scale.cpu().double().repeat_interleave(group, -1)
    assert worst(q.float() * scale.repeat_interleave(group, -1), y,
                 (2.0 ** -4 + 128 * U32) * y.abs() + 2.0 ** -10 * s) <= 1


def test_norm_of_zero_rows_and_of_rows_of_zeros():
    w = torch.ones(64, device="cuda")
    x = torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16)
    out, r, q, scale = binding.ida_rmsnorm(x, w, residual=x.clone(), group=32)
    e = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    none, _, _, _ = binding.ida_rmsnorm(e, w)
    g = binding.ida_rmsnorm_backward(e, w, e)
    _done()
    assert out is None and not r.any() and not q.float().any() and bool((scale == 1).all())
    assert none.numel() == 0 and not g["w"].any()


def test_norm_in_place_on_the_stream_and_on_the_input():
    x, res, w = _inputs(21, 256, "bf16", True)
    ref, r0, _, _ = binding.ida_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda())
    for into in ("x", "residual"):
        dx, dr = x.cuda(), res.cuda()
        out, r, _, _ = binding.ida_rmsnorm(dx, w.cuda(), residual=dr, res_out=dx if into == "x" else dr)
        _done()
        assert torch.equal(out, ref) and torch.equal(r, r0)
        assert torch.equal(dx if into == "x" else dr, r0)


def test_norm_takes_leading_dimensions_and_keeps_rows_apart():
    """Rows of any leading shape; a row of NaN or infinities changes no other."""
    x, res, w = _inputs(24, 128, "bf16", True)
    ref, _, q0, s0 = binding.ida_rmsnorm(x.cuda().view(2, 12, 128), w.cuda(), residual=res.cuda().view(2, 12, 128), group=64,
                                         out=torch.empty(2, 12, 128, device="cuda", dtype=torch.bfloat16))
    assert q0.shape == (2, 12, 128) and s0.shape == (2, 12, 2)
    x[5, 3], x[9, 7] = float("nan"), float("inf")
    out, _, q, s = binding.ida_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), group=64,
                                       out=torch.empty(24, 128, device="cuda", dtype=torch.bfloat16))
    _done()
    keep = [i for i in range(24) if i not in (5, 9)]
    assert torch.equal(out[keep], ref.view(24, 128)[keep])
    assert torch.equal(s[keep], s0.view(24, 2)[keep])
    assert torch.equal(q[keep].float(), q0.view(24, 128)[keep].float())


# (rows, D, dtype, dres)
BWDS = [(1, 8, "bf16", True), (5, 768, "bf16", False), (9, 2048, "f32", True), (700, 768, "bf16", True),
        (3000, 64, "f32", False), (13, 4104, "f32", True), (6, 8192, "bf16", True), (20, 8192, "f32", True),
        (2, 1000, "bf16", True), (4, 5000, "bf16", False)]


@pytest.mark.parametrize("case", BWDS, ids=str)
def test_norm_backward(case):
    rows, D, dtype, has = case
    r, dres, w = _inputs(rows, D, dtype, has, seed=4)
    dy = torch.randn(rows, D, generator=sc.gen(5)).to(sc.DT[dtype])
    args = (r.cuda(), w.cuda(), dy.cuda())
    g = binding.ida_rmsnorm_backward(*args, dres=None if dres is None else dres.cuda(), eps=EPS)
    again = binding.ida_rmsnorm_backward(*args, dres=None if dres is None else dres.cuda(), eps=EPS)
    _done()
    assert torch.equal(g["x"], again["x"]) and torch.equal(g["w"], again["w"])
    r64, w64, dy64 = r.double(), w.double(), dy.double()
    rx, rw = orc.grads(lambda a, b: orc.rmsnorm(a, b, EPS), [r64, w64], dy64)
    inv = 1 / torch.sqrt((r64 * r64).mean(-1, keepdim=True) + EPS)
    gw = (dy64 * w64).abs()
    size = inv * (gw + r64.abs() * inv * inv * (gw * r64.abs()).mean(-1, keepdim=True))
    if dres is not None:
        rx, size = rx + dres.double(), size + dres.double().abs()
    assert worst(g["x"], rx, HALF[dtype] * rx.abs() + 2 * 64 * U32 * size) <= 1
    # rows add up within a block (rows / 1216 of them), then over at most 1216 blocks in 32 parts
    n = 64 + rows // 1216 + 1216 // 32 + 8
    assert worst(g["w"], rw, n * U32 * (dy64 * r64 * inv).abs().sum(0)) <= 1


def test_norm_backward_in_place():
    r, dres, w = _inputs(50, 768, "bf16", True, seed=6)
    dy = torch.randn(50, 768, generator=sc.gen(7)).to(torch.bfloat16)
    ref = binding.ida_rmsnorm_backward(r.cuda(), w.cuda(), dy.cuda(), dres=dres.cuda())
    for which in (0, 1):
        a, b = dy.cuda(), dres.cuda()
        g = binding.ida_rmsnorm_backward(r.cuda(), w.cuda(), a, dres=b, dx=(a, b)[which])
        _done()
        assert torch.equal(g["x"], ref["x"]) and torch.equal(g["w"], ref["w"])


@pytest.mark.parametrize("back", [False, True])
def test_norm_captured_and_replayed(back):
    x, res, w = _inputs(40, 768, "bf16", True)
    x, res, w = x.cuda(), res.cuda(), w.cuda()

    def call():
        if back:
            g = binding.ida_rmsnorm_backward(x, w, res)
            return [g["x"], g["w"]]
        out, r, q, s = binding.ida_rmsnorm(x, w, residual=res, group=128)
        return [r, q.view(torch.uint8), s]

    ref = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for t in got:
        t.zero_()
    graph.replay()
    _done()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_rows_past_32_bits():
    rows, D = (1 << 19) + 3, 8192
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator().manual_seed(5)
    last = torch.randn(5, D, generator=g).bfloat16().cuda()
    w = torch.randn(D, generator=g).cuda()
    x = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    x[-5:] = last
    out, _, _, _ = binding.ida_rmsnorm(x, w)
    want, _, _, _ = binding.ida_rmsnorm(last, w)
    assert torch.equal(out[-5:], want) and not out[:-5].any()
    _, _, q, scale = binding.ida_rmsnorm(x, w, group=128)
    _, _, wq, ws = binding.ida_rmsnorm(last, w, group=128)
    assert torch.equal(q[-5:].view(torch.uint8), wq.view(torch.uint8)) and torch.equal(scale[-5:], ws)
    del q, scale
    dx = binding.ida_rmsnorm_backward(x, w, out)["x"]
    assert torch.equal(dx[-5:], binding.ida_rmsnorm_backward(last, w, want)["x"])
