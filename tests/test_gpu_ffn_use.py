"""The feed-forward block and the 8-bit products as they are used: in a decoder layer, in slices of wider rows, on other
streams, captured and replayed, with workspaces of any contents, far and many rows, odd values."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, inputs
from tests import ffn_cases as fc
from tests.ssm_cases import DT, HALF, gen, worst

pytestmark = pytest.mark.gpu
NAMES = ("x", "w_gate", "w_up", "w_down")


def _done():
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0


def _inputs(T, D, F, dtype, seed=0):
    return [t.cuda() for t in (fc.rows(T, D, dtype, seed), *fc.weights(D, F, dtype, seed + 1))]


def _operand(T, K, block_rows, seed):
    return [t.cuda() for t in fc.quantised(torch.randn(T, K, generator=gen(seed)), block_rows)]


def _calls(T, dtype, D=256, F=384):
    """{name: (call, outputs' names)}: every entry point with outputs of its own."""
    x, wg, wu, wd = _inputs(T, D, F, dtype, 3)
    dy = fc.rows(T, D, dtype, 9).cuda()
    acts = binding.ida_ffn(x, wg, wu, wd, acts=True)[1]
    a, b, c = _operand(T, D, 1, 4), _operand(F, D, 128, 5), _operand(F, D, 128, 6)
    return {"ffn": lambda: list(binding.ida_ffn(x, wg, wu, wd, acts=True)),
            "ffn backward": lambda: list(binding.ida_ffn_backward(x, wg, wu, wd, acts, dy).values()),
            "quant rows": lambda: list(binding.ida_quant_e4m3(x)), "quant blocks": lambda: list(binding.ida_quant_e4m3(wg, rows=128)),
            "gemm": lambda: [binding.ida_gemm_e4m3(*a, *b, dtype=DT[dtype])], "glu": lambda: list(binding.ida_glu_e4m3(*a, *b, *c))}


def _same(got, want):
    return all(torch.equal(g.float(), w.float()) for g, w in zip(got, want, strict=True))


CALLS = ["ffn", "ffn backward", "quant rows", "quant blocks", "gemm", "glu"]


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed(name, T):
    call = _calls(T, "bf16")[name]
    want = [t.clone() for t in call()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        for t in got:
            t.view(torch.uint8).fill_(127)
        graph.replay()
        _done()
        assert _same(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", CALLS)
def test_on_another_stream_and_again(name, dtype):
    call = _calls(200, dtype)[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    _done()
    assert _same(got, want) and _same(call(), want)


def test_two_calls_at_once():
    one, two = _calls(700, "bf16"), _calls(40, "bf16")
    want = {k: ([t.clone() for t in one[k]()], [t.clone() for t in two[k]()]) for k in CALLS}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for k in CALLS:
            for m in CALLS:
                got = one[k]()
                with torch.cuda.stream(side):
                    other = two[m]()
                _done()
                assert _same(got, want[k][0]) and _same(other, want[m][1])


def test_beside_the_mixers_on_another_stream():
    """The block and the 8-bit products while the mixer's and the selective mixer's prompts run on another stream."""
    p = binding.params_to_device(inputs.make_params(H=4, R=64, d=64, M=64, W=4, seed=3))
    qkv = inputs.make_qkv(2, 1024, 4, 64, 64, "bf16", 4, device="cuda")
    sp = {"a_log": torch.zeros(4, device="cuda"), "dt_bias": torch.full((4,), -4.0, device="cuda"), "D": torch.ones(4, device="cuda")}
    bc = torch.randn(2, 1024, 1, 64, generator=gen(5)).bfloat16().cuda()
    dt = torch.randn(2, 1024, 4, generator=gen(6)).bfloat16().cuda()

    def mixers():
        return [binding.ida_forward(*qkv, p)[0], binding.ida_ssm_scan(qkv[2], bc, bc, dt, sp)[0]]

    calls = _calls(900, "bf16")
    want, other = {k: [t.clone() for t in calls[k]()] for k in CALLS}, [t.clone() for t in mixers()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in CALLS:
        with torch.cuda.stream(side):
            mixed = [mixers() for _ in range(3)]
        got = [calls[k]() for _ in range(3)]
        _done()
        assert all(_same(g, want[k]) for g in got) and all(_same(m, other) for m in mixed), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,F", [(3, 64, 136), (200, 264, 520), (600, 520, 1032)])
def test_workspaces_of_any_contents_and_two_graphs_over_one(T, D, F, dtype):
    args = _inputs(T, D, F, dtype)
    dy = fc.rows(T, D, dtype, 8).cuda()
    code = binding._dtype_code(args[0])
    want, acts = binding.ida_ffn(*args, acts=True)
    grads = binding.ida_ffn_backward(*args, acts, dy)
    n = max(binding.ida_ffn_workspace_bytes(T, D, F, code), binding.ida_ffn_backward_workspace_bytes(T, D, F, code))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN in either type
    assert torch.equal(binding.ida_ffn(*args, workspace=ws)[0], want)
    ws.fill_(255)
    assert _same(binding.ida_ffn_backward(*args, acts, dy, workspace=ws).values(), grads.values())
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        out = binding.ida_ffn(*args, workspace=ws)[0]
    with torch.cuda.graph(graphs[1]):
        g = binding.ida_ffn_backward(*args, acts, dy, workspace=ws)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    _done()
    assert torch.equal(out, want) and _same(g.values(), grads.values())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [6, 120, 700])
def test_slices_of_wider_rows_and_leading_dimensions(T, dtype):
    D, F = 264, 392
    x, wg, wu, wd = _inputs(T, D, F, dtype)
    wide = torch.full((T, D + 24), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 8:8 + D] = x
    want, acts = binding.ida_ffn(x, wg, wu, wd, acts=True)
    dy = fc.rows(T, D, dtype, 5).cuda()
    grads = binding.ida_ffn_backward(x, wg, wu, wd, acts, dy)
    for view, lead in ((wide[:, 8:8 + D], (T,)), (wide.view(2, T // 2, -1)[..., 8:8 + D], (2, T // 2)), (x.view(2, 1, T // 2, D), (2, 1, T // 2))):
        out, a = binding.ida_ffn(view, wg, wu, wd, acts=True)
        assert out.shape == (*lead, D) and a.shape == (3, *lead, F)
        assert torch.equal(out.reshape(T, D), want) and torch.equal(a.reshape(3, T, F), acts)
        g = binding.ida_ffn_backward(view, wg, wu, wd, acts.view(3, *lead, F), dy.view(*lead, D))
        assert g["x"].shape == (*lead, D) and _same([t.reshape(w.shape) for t, w in zip(g.values(), grads.values())], grads.values())
    D = 256  # a multiple of 16 for e4m3
    q, s = binding.ida_quant_e4m3(wide[:, 8:8 + D])
    q2, s2 = binding.ida_quant_e4m3(wide[:, 8:8 + D].contiguous().view(2, 1, T // 2, D))
    assert q2.shape == (2, 1, T // 2, D) and s2.shape == (2, 1, T // 2, 2)
    assert _same([q2.view(T, D), s2.view(T, 2)], [q, s])
    b, c = _operand(144, D, 128, 5), _operand(144, D, 128, 6)
    assert torch.equal(binding.ida_gemm_e4m3(q2, s2, *b).view(T, 144), binding.ida_gemm_e4m3(q, s, *b))
    assert _same([t.reshape(w.shape) for t, w in zip(binding.ida_glu_e4m3(q2, s2, *b, *c), binding.ida_glu_e4m3(q, s, *b, *c))],
                 binding.ida_glu_e4m3(q, s, *b, *c))
    w1, w2 = binding.ida_quant_e4m3(wide[:, 8:8 + D], rows=128), binding.ida_quant_e4m3(wide[:, 8:8 + D].contiguous(), rows=128)
    assert _same(w1, w2)
    _done()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(dtype):
    x, wg, wu, wd = _inputs(4, 64, 128, dtype)
    x = x[:0]
    out, acts = binding.ida_ffn(x, wg, wu, wd, acts=True)
    assert out.shape == (0, 64) and acts.shape == (3, 0, 128)
    g = binding.ida_ffn_backward(x, wg, wu, wd, acts, x)
    assert g["x"].shape == (0, 64) and all(bool((g[k] == 0).all()) for k in NAMES[1:])
    q, s = binding.ida_quant_e4m3(x)
    b = _operand(136, 64, 128, 3)
    assert s.shape == (0, 1) and binding.ida_gemm_e4m3(q, s, *b).shape == (0, 136)
    c = _operand(144, 64, 128, 3)
    assert [t.shape for t in binding.ida_glu_e4m3(q, s, *c, *c)] == [(0, 144), (0, 2)]
    _done()


@pytest.mark.parametrize("T,D,F", [(5, 64, 144), (131, 72, 136), (300, 264, 1040), (290, 64, 2064)])
def test_outputs_stay_inside_their_tensors(T, D, F):
    """Guard bands around every output and workspace, rows behind the last and columns behind the last among them."""
    raws = []

    def guarded(shape, dtype):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        n = t.numel() * t.element_size()
        raw = torch.full((n + 131072,), 77, dtype=torch.uint8, device="cuda")
        raws.append((raw, n))
        return raw[65536:65536 + n].view(dtype).view(shape)

    for dtype in ("bf16", "f32"):
        x, wg, wu, wd = _inputs(T, D, F, dtype)
        dt, code = x.dtype, binding._dtype_code(x)
        acts = guarded((3, T, F), dt)
        binding.ida_ffn(x, wg, wu, wd, out=guarded((T, D), dt), acts=acts,
                        workspace=guarded((binding.ida_ffn_workspace_bytes(T, D, F, code),), torch.uint8))
        binding.ida_ffn_backward(x, wg, wu, wd, acts, x, grads={k: guarded(t.shape, dt) for k, t in zip(NAMES, (x, wg, wu, wd))},
                                 workspace=guarded((binding.ida_ffn_backward_workspace_bytes(T, D, F, code),), torch.uint8))
    K = F // 16 * 16
    x = torch.randn(T, K, device="cuda")
    for block_rows in (1, 128):
        binding.ida_quant_e4m3(x, rows=block_rows, q=guarded((T, K), fc.E4M3), scale=guarded((-(-T // block_rows), -(-K // 128)), torch.float32))
    a, b, c = binding.ida_quant_e4m3(x), _operand(D, K, 128, 3), _operand(80, K, 128, 4)
    for dt in (torch.bfloat16, torch.float32):
        binding.ida_gemm_e4m3(*a, *b, out=guarded((T, D), dt))
    binding.ida_glu_e4m3(*a, *c, *c, q=guarded((T, 80), fc.E4M3), scale=guarded((T, 1), torch.float32))
    _done()
    for raw, n in raws:
        assert bool((raw[:65536] == 77).all()) and bool((raw[65536 + n:] == 77).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [7, 200, 600])
def test_a_row_that_is_not_finite_stays_alone(T, dtype):
    D, F = 264, 392
    x, wg, wu, wd = _inputs(T, D, F, dtype)
    dy = fc.rows(T, D, dtype, 4).cuda()
    want, acts = binding.ida_ffn(x, wg, wu, wd, acts=True)
    dx = binding.ida_ffn_backward(x, wg, wu, wd, acts, dy)["x"]
    bad, keep = x.clone(), torch.arange(T, device="cuda") != 3
    for v in (float("nan"), float("inf")):
        bad[3, 5] = v
        out, a = binding.ida_ffn(bad, wg, wu, wd, acts=True)
        assert torch.equal(out[keep], want[keep]) and not bool(torch.isfinite(out[3]).all())
        got = binding.ida_ffn_backward(bad, wg, wu, wd, a, dy)["x"]
        assert torch.equal(got[keep], dx[keep])
    K = 256
    q, s = binding.ida_quant_e4m3(x[:, :K].contiguous())
    bad = x[:, :K].contiguous()
    bad[3, 5] = float("nan")
    qn, sn = binding.ida_quant_e4m3(bad)
    at = torch.ones_like(q, dtype=torch.bool)
    at[3, 5] = False
    assert bool(torch.isnan(qn.float()[3, 5])) and torch.equal(qn.float()[at], q.float()[at]) and torch.equal(s[keep], sn[keep])
    b, c = _operand(144, K, 128, 5), _operand(144, K, 128, 6)
    assert torch.equal(binding.ida_gemm_e4m3(qn, sn, *b)[keep], binding.ida_gemm_e4m3(q, s, *b)[keep])
    assert _same([t[keep] for t in binding.ida_glu_e4m3(qn, sn, *b, *c)], [t[keep] for t in binding.ida_glu_e4m3(q, s, *b, *c)])
    _done()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 150])
def test_gates_far_out(T, dtype):
    """Gates of +-200 and beyond: silu is the gate itself or 0, its slope 1 or 0, where e^-g passes fp32."""
    D, F = 64, 136
    x, wg, wu, wd = [t.cpu() for t in _inputs(T, D, F, dtype)]
    x = (x.float() * 200).to(x.dtype)
    dy = fc.rows(T, D, dtype, 4)
    ref = fc.forward_ref(x, wg, wu, wd, dtype)
    out, acts = binding.ida_ffn(*[t.cuda() for t in (x, wg, wu, wd)], acts=True)
    for name, got in zip(("out", "g", "u", "h"), (out, *acts)):
        assert worst(got, *ref[name]) <= 1, name
    kept = torch.stack([ref[k][0] for k in "guh"]).to(DT[dtype])
    got = binding.ida_ffn_backward(*[t.cuda() for t in (x, wg, wu, wd, kept, dy)])
    for name, (v, e) in fc.backward_ref(x, wg, wu, wd, kept, dy, dtype).items():
        assert worst(got[name], v, e) <= 1, name


@pytest.mark.parametrize("T", [4, 200, 1200])
def test_fp32_of_any_size(T):
    """Values whose parts reach from 2^-100 to 2^100: products are exact to fp32 whatever their size."""
    D, F = 256, 512
    x, wg, wu, wd = [t.cpu() for t in _inputs(T, D, F, "f32")]
    for up in (100, -80):
        a, b = x * 2.0 ** up, [t * 2.0 ** -up for t in (wg, wu)]
        ref = fc.forward_ref(a, *b, wd, "f32")
        out, acts = binding.ida_ffn(*[t.cuda() for t in (a, *b, wd)], acts=True)
        for name, got in zip(("out", "g", "u", "h"), (out, *acts)):
            assert worst(got, *ref[name]) <= 1, (name, up)


def test_scales_of_any_size():
    """Groups from the least subnormal to the largest fp32 numbers, and their products."""
    x = torch.randn(40, 512, generator=gen(3))
    size = torch.tensor([2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -120, 2.0 ** -101, 2.0 ** -90, 2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 125])
    x = (x.double() * size.double().repeat_interleave(4)[:, None]).clamp(-3.4e38, 3.4e38).float()
    for block_rows in (1, 128):
        for rows in ([x[4 * i:4 * i + 4] for i in range(10)] if block_rows == 128 else [x]):
            q, s = (t.cpu() for t in binding.ida_quant_e4m3(rows.cuda(), rows=block_rows))
            v = fc.values(q, s, block_rows)
            top = rows.double().abs().view(-1, 4, 128) if block_rows == 128 else rows.double().abs().view(rows.shape[0], 4, 128)
            top = top.amax((0, 2), keepdim=True) if block_rows == 128 else top.amax(2, keepdim=True)
            sd = s.double().view(-1, 4, 1) if block_rows == 1 else s.double().view(1, 4, 1)
            assert bool((sd >= top / 448 * (1 - 2.0 ** -24)).all() or (top == 0).any())
            # the scale is off by half a step of fp32, or rounded up to a subnormal; the quotient by a division
            half = 2.0 ** -4 * rows.double().abs() + 2.0 ** -10 * (1 + 2.0 ** -20) * sd.expand(-1, -1, 128).reshape(-1, 512)
            assert bool(((v - rows.double()).abs() <= half * (1 + 2.0 ** -20)).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_past_32_bits(dtype):
    """Rows 2^26 elements apart, the last ones past element 2^32: the results of dense rows."""
    T, D, F, ld = 70, 256, 384, 1 << 26
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 20 GB")
    x, wg, wu, wd = _inputs(T, D, F, dtype)
    far = torch.empty(T * ld, dtype=x.dtype, device="cuda").as_strided((T, D), (ld, 1))
    far.copy_(x)
    dy = fc.rows(T, D, dtype, 4).cuda()
    want, acts = binding.ida_ffn(x, wg, wu, wd, acts=True)
    got, a = binding.ida_ffn(far, wg, wu, wd, acts=True)
    assert torch.equal(got, want) and torch.equal(a, acts)
    assert _same(binding.ida_ffn_backward(far, wg, wu, wd, acts, dy).values(), binding.ida_ffn_backward(x, wg, wu, wd, acts, dy).values())
    assert torch.equal(binding.ida_ffn(far[60:68], wg, wu, wd)[0], binding.ida_ffn(x[60:68].contiguous(), wg, wu, wd)[0])
    for block_rows in (1, 128):
        assert _same(binding.ida_quant_e4m3(far, rows=block_rows), binding.ida_quant_e4m3(x, rows=block_rows))
    _done()


def test_many_rows():
    """More rows than 2^16 tiles of 32, and outputs past 2^31 elements: the last rows are those of a call of their own."""
    T, D, F = 2200000, 16, 1008
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 30 GB")
    x = torch.randn(T, D, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    _, wg, wu, wd = _inputs(4, D, F, "bf16")
    out, acts = binding.ida_ffn(x, wg, wu, wd, acts=True)
    want, a = binding.ida_ffn(x[-300:].contiguous(), wg, wu, wd, acts=True)
    # 300 rows' projection back is shared over pairs of SMs, all rows' is not: equal but for the order of sums
    assert torch.equal(acts[:, -300:], a)
    ref = fc.forward_ref(*[t.cpu() for t in (x[-300:], wg, wu, wd)], "bf16")["out"]
    assert worst(out[-300:], *ref) <= 1 and worst(want, *ref) <= 1
    q, s = binding.ida_quant_e4m3(x)
    b, c = _operand(F, D, 128, 5), _operand(F, D, 128, 6)
    h = binding.ida_glu_e4m3(q, s, *b, *c)
    assert _same([t[-300:] for t in h], binding.ida_glu_e4m3(q[-300:].contiguous(), s[-300:].contiguous(), *b, *c))
    d = _operand(D, F, 128, 7)
    got = binding.ida_gemm_e4m3(*h, *d)
    ref = binding.ida_gemm_e4m3(*[t[-300:].contiguous() for t in h], *d)
    err = fc.product_err(F) * (fc.values(*[t[-300:].cpu() for t in h], 1).abs() @ fc.values(*[t.cpu() for t in d], 128).abs().t())
    assert worst(got[-300:], ref.cpu().double(), 2 * err + 2 * HALF["bf16"] * ref.cpu().double().abs()) <= 1
    _done()


def test_gradients_agree_with_differences():
    """Central differences of L = sum dout * out in fp32, out in 64 bits: h^2 / 6 times a third derivative is far below."""
    T, D, F = 20, 64, 72
    x, wg, wu, wd = [t.cpu() for t in _inputs(T, D, F, "f32")]
    dy = fc.rows(T, D, "f32", 4)
    acts = binding.ida_ffn(*[t.cuda() for t in (x, wg, wu, wd)], acts=True)[1]
    g = binding.ida_ffn_backward(*[t.cuda() for t in (x, wg, wu, wd)], acts, dy.cuda())
    args = [t.double() for t in (x, wg, wu, wd)]

    def loss(k, d):
        a = list(args)
        a[k] = a[k] + d
        gate, up = a[0] @ a[1].t(), a[0] @ a[2].t()
        return ((gate * torch.sigmoid(gate) * up) @ a[3].t() * dy.double()).sum()

    for k, name in enumerate(NAMES):
        d = torch.randn(args[k].shape, generator=gen(20 + k), dtype=torch.float64)
        want = (loss(k, 1e-5 * d) - loss(k, -1e-5 * d)) / 2e-5
        got = (g[name].cpu().double() * d).sum()
        # the gradients' own error is below 2^-17 of the sums of magnitudes; the difference's below 1e-8
        size = (g[name].cpu().double() * d).abs().sum()
        assert abs(got - want) <= 2.0 ** -15 * size, name


def test_a_layers_second_half_in_8_bits():
    """Norm with e4m3 output, gated projection, projection back, added to the stream by the next norm; for a prompt
    and for its next rows.  Each step against 64 bits on what it was given."""
    D, F = 256, 640
    norm_w = torch.ones(D, device="cuda")
    wg, wu, wd = (t.cuda() for t in fc.weights(D, F, "f32", 3))
    qg, qu, qd = (binding.ida_quant_e4m3(w, rows=128) for w in (wg, wu, wd))
    for T in (300, 4, 1):
        x, stream = (torch.randn(2, T, D, generator=gen(T + i)).bfloat16().cuda() for i in (0, 1))
        _, r, q, s = binding.ida_rmsnorm(x, norm_w, residual=stream, group=128)
        hq, hs = binding.ida_glu_e4m3(q, s, *qg, *qu)
        out = binding.ida_gemm_e4m3(hq, hs, *qd)
        y, r2, _, _ = binding.ida_rmsnorm(out, norm_w, residual=r)
        _done()
        assert out.shape == x.shape and y.shape == x.shape
        flat = lambda t: t.reshape(2 * T, -1).cpu()  # noqa: E731
        h, e = fc.glu_ref(fc.values(flat(q), flat(s), 1), *(fc.values(a.cpu(), b.cpu(), 128) for a, b in (qg, qu)))
        got = fc.values(flat(hq), flat(hs), 1)
        sc = flat(hs).double().repeat_interleave(128, 1)[:, :F]
        assert worst(got, h, 1.07 * e + (2.0 ** -4 + 2.0 ** -21) * h.abs() + 2.0 ** -10 * sc) <= 1
        v, e = fc.product_ref(got, fc.values(qd[0].cpu(), qd[1].cpu(), 128))
        assert worst(flat(out), v, e + HALF["bf16"] * v.abs()) <= 1
        # and of the block in full precision: 8 bits cost what they cost (a relative 2^-4 a value at worst, three times over)
        n = binding.ida_rmsnorm(x, norm_w, residual=stream)[0]
        full = binding.ida_ffn(n.float(), wg, wu, wd)[0]
        assert float((out.float() - full).norm() / full.norm()) <= 4 * 2.0 ** -4
        assert torch.equal(r2, (out.float() + r.float()).bfloat16())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_the_second_half_of_a_layer(dtype):
    """Norm, block and their gradients chained: dx of the block is the norm's dy, each against 64 bits on what it was given."""
    T, D, F = 260, 128, 344
    x, wg, wu, wd = _inputs(T, D, F, dtype)
    w = torch.ones(D, device="cuda")
    n, r, _, _ = binding.ida_rmsnorm(x, w, residual=fc.rows(T, D, dtype, 5).cuda())
    out, acts = binding.ida_ffn(n, wg, wu, wd, acts=True)
    dout = fc.rows(T, D, dtype, 6).cuda()
    g = binding.ida_ffn_backward(n, wg, wu, wd, acts, dout)
    gn = binding.ida_rmsnorm_backward(r, w, g["x"], dres=dout)
    _done()
    ref = fc.forward_ref(*[t.cpu() for t in (n, wg, wu, wd)], dtype)
    assert worst(out, *ref["out"]) <= 1
    for name, (v, e) in fc.backward_ref(*[t.cpu() for t in (n, wg, wu, wd, acts, dout)], dtype).items():
        assert worst(g[name], v, e) <= 1, name
    rd, dn = r.cpu().double(), g["x"].cpu().double()
    rms = (rd.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    dx = (dn - rd / rms * (dn * rd / rms).mean(-1, keepdim=True)) / rms + dout.cpu().double()
    size = (dn.abs() + (rd / rms).abs() * (dn * rd / rms).abs().mean(-1, keepdim=True)) / rms + dout.cpu().double().abs()
    assert worst(gn["x"], dx, HALF[dtype] * dx.abs() + (D + 10) * 2.0 ** -24 * size) <= 1
