"""GPU parity of the selective mixer where a call divides its work: sequences split into segments and
parts of them, groups whose heads one CTA takes in turn, several passes of the blocks that sum the
convolution's gradients.  Each case proves from the workspace it asks for that it is divided so.

Bounds as in ``test_gpu_ssm.py``.
"""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from oracle import ida_ssm as orc
from tests import ssm_cases as sc
from tests.ssm_cases import HALF, U32, worst
from tests.test_gpu_ssm import _done, _on_gpu, _scan_bounds, _scan_inputs, _scan_ref
from tests.test_gpu_ssm_extremes import check_scan_gradients

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


# (B, N, H, d, G, M, dtype, state, fast): bf16 sequences behind 1024 positions on idle SMs
SPLIT_SCANS = [
    (1, 1100, 4, 32, 1, 16, "bf16", True, False),    # a chunk a segment
    (3, 1700, 4, 64, 2, 64, "bf16", False, False),   # segments of several chunks
    (16, 2304, 4, 8, 1, 8, "bf16", True, False),     # two segments, states of parts of them
    (1, 1300, 2, 128, 1, 128, "bf16", True, False),  # the widest tiles: one CTA an SM
    (1, 1200, 2, 256, 2, 24, "bf16", True, False),   # two slices of channels
    (2, 1500, 3, 72, 1, 72, "bf16", False, True),    # decays that underflow within a few positions
    (1, 33000, 1, 8, 1, 8, "bf16", True, False),     # more chunks than segments are tried
]


@pytest.mark.parametrize("case", SPLIT_SCANS, ids=str)
def test_scan_in_segments(case):
    B, N, H, d, G, M, dtype, state, _ = case
    p, row, s, C = _scan_inputs(*case)
    assert binding.ida_ssm_scan_workspace_bytes(B, H, N, d, G, M, binding.IDA_BF16) > 0
    args = (*_on_gpu(row, C, H, d, G, M), sc.cuda(p))
    given = None if s is None else s.cuda()
    y, X = binding.ida_ssm_scan(*args, state_in=given, final_state=True)
    z, none = binding.ida_ssm_scan(*args, state_in=given)
    whole = torch.empty(0, dtype=torch.uint8, device="cuda")  # no workspace: the sequence in one piece
    y1, X1 = binding.ida_ssm_scan(*args, state_in=given, final_state=True, workspace=whole)
    _done()
    ry, rX = _scan_ref(row, C, H, d, G, M, p, s)
    ya, Xa = _scan_ref(row, C, H, d, G, M, p, s, absolute=True)
    by, bX = _scan_bounds(dtype, N, ry, ya, Xa)
    for got in (y, z, y1):
        assert worst(got, ry, by) <= 1
    for got in (X, X1):
        assert worst(got, rX, bX) <= 1
    assert none is None


@pytest.mark.parametrize("case", SPLIT_SCANS[:4], ids=str)
def test_outputs_do_not_depend_on_whether_the_final_state_is_wanted(case):
    B, N, H, d, G, M = case[:6]
    p, row, s, C = _scan_inputs(*case)
    args = (*_on_gpu(row, C, H, d, G, M), sc.cuda(p))
    given = None if s is None else s.cuda()
    y, _ = binding.ida_ssm_scan(*args, state_in=given, final_state=True)
    z, _ = binding.ida_ssm_scan(*args, state_in=given)
    _done()
    assert torch.equal(y, z)


# (B, N, H, d, G, M): a row's chunks fill the SMs, so that one CTA takes all heads of a group
SHARED_HEADS = [
    (152, 20, 70, 8, 1, 16),   # more heads than two batches of rates
    (160, 64, 3, 16, 1, 16),
    (40, 260, 4, 72, 2, 40),   # chunks of 128 positions, two groups, wide heads
    (76, 70, 3, 8, 1, 72),     # chunks of 64 positions, G made again for every head
    (50, 130, 2, 72, 1, 128),
]


def _backward_floats_of_one_part(B, N, H, d, G, M):
    """Workspace of gradients whose groups are not divided: no partial rows of db and dc."""
    q = 128 if M <= 64 else 64
    chunks = B * H * ((N + q - 1) // q)
    return 2 * chunks * M * d + 16 * chunks + (chunks + 3) // 4 * 4


@pytest.mark.parametrize("case", SHARED_HEADS, ids=str)
def test_scan_backward_with_the_heads_of_a_group_in_one_block(case):
    B, N, H, d, G, M = case
    assert binding.ida_ssm_scan_backward_workspace_bytes(B, H, N, d, G, M, binding.IDA_BF16) == \
        4 * _backward_floats_of_one_part(*case)
    p, row, _, C = _scan_inputs(*case, "bf16", False, False)
    dy = torch.randn(B, N, H, d, generator=sc.gen(11)).bfloat16()
    g = binding.ida_ssm_scan_backward(*_on_gpu(row, C, H, d, G, M), sc.cuda(p), dy.cuda())
    _done()
    check_scan_gradients(g, row, C, H, d, G, M, p, dy)


def test_conv_backward_over_several_passes_of_the_blocks():
    """One block for each 128 of the channels, which takes at most 8 strips of 64 positions at a time:
    600 positions are several passes."""
    B, N, C, W = 2, 300, 19584, 4
    assert binding.ida_ssm_conv_backward_workspace_bytes(B, N, C, W) == 4 * (W + 1) * C and B * N > 8 * 64
    p, row = sc.params(1, C, W, 3), sc.rows(B, N, C, 5, "bf16", 4)
    dout = torch.randn(B, N, C, generator=sc.gen(8)).bfloat16()
    g = binding.ida_ssm_conv_backward(row.cuda()[..., :C], dout.cuda(), p["conv_w"].cuda(), p["conv_b"].cuda())
    again = binding.ida_ssm_conv_backward(row.cuda()[..., :C], dout.cuda(), p["conv_w"].cuda(), p["conv_b"].cuda())
    _done()
    assert all(torch.equal(g[k], again[k]) for k in g)
    x, w, b = row[..., :C].double(), p["conv_w"].double(), p["conv_b"].double()
    rx, rw, rb = orc.grads(lambda *v: orc.conv(*v)[0], [x, w, b], dout.double())
    rows = torch.cat([torch.zeros(B, W - 1, C, dtype=torch.float64), x], 1)
    pre = b.abs() + sum(w[:, j].abs() * rows[:, j:j + N].abs() for j in range(W))
    eg = dout.double().abs() * U32 * (0.5 * (W + 2) * pre + 16 * (1 + pre))
    ga = 1.1 * dout.double().abs()
    ex = torch.zeros_like(x)
    for j in range(W):
        k = W - 1 - j
        ex[:, :N - k] += w[:, j].abs() * (eg + W * U32 * ga)[:, k:]
    assert worst(g["x"], rx, HALF["bf16"] * rx.abs() + ex) <= 1
    n = 64 + 8 + B * N // 512 + 8
    ew = torch.stack([((eg + n * U32 * ga) * rows[:, j:j + N].abs()).sum((0, 1)) for j in range(W)], -1)
    assert worst(g["conv_w"], rw, ew + U32 * rw.abs()) <= 1
    assert worst(g["conv_b"], rb, (eg + n * U32 * ga).sum((0, 1)) + U32 * rb.abs()) <= 1


def test_heads_of_one_block_keep_their_non_finite_values():
    """A NaN in one head's x and an infinite step size reach that head's gradients and its group's db and dc
    only, also where one CTA takes the head before and the heads behind."""
    B, N, H, d, G, M = 160, 64, 6, 16, 2, 16
    assert binding.ida_ssm_scan_backward_workspace_bytes(B, H, N, d, G, M, binding.IDA_BF16) == \
        4 * _backward_floats_of_one_part(B, N, H, d, G, M)
    p, row, _, C = _scan_inputs(B, N, H, d, G, M, "bf16", False, False)
    dy = torch.randn(B, N, H, d, generator=sc.gen(11)).bfloat16().cuda()
    g0 = binding.ida_ssm_scan_backward(*_on_gpu(row, C, H, d, G, M), sc.cuda(p), dy)
    row[:, 30, d + 3] = float("nan")  # x of head 1
    row[:, 20, C + 1] = float("inf")  # dt of head 1
    g1 = binding.ida_ssm_scan_backward(*_on_gpu(row, C, H, d, G, M), sc.cuda(p), dy)
    _done()
    for h in (0, 2, 3, 4, 5):
        assert torch.equal(g0["x"][:, :, h], g1["x"][:, :, h]) and torch.equal(g0["dt"][:, :, h], g1["dt"][:, :, h])
        assert all(torch.equal(g0[k][h], g1[k][h]) for k in ("a_log", "dt_bias", "D"))
    assert torch.equal(g0["b"][:, :, 1], g1["b"][:, :, 1]) and torch.equal(g0["c"][:, :, 1], g1["c"][:, :, 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_at_once_on_two_streams(dtype):
    """Split prompts and gradients of two problems beside each other give what each gives alone."""
    B, N, H, d, G, M = 2, 1300, 3, 64, 1, 64
    work = []
    for seed in (5, 25):
        p, row, s, C = _scan_inputs(B, N, H, d, G, M, dtype, True, False, seed)
        args, dp, given = _on_gpu(row, C, H, d, G, M), sc.cuda(p), s.cuda()
        dy = torch.randn(B, N, H, d, generator=sc.gen(seed)).to(sc.DT[dtype]).cuda()

        def call(args=args, dp=dp, given=given, dy=dy):
            out = list(binding.ida_ssm_scan(*args, dp, state_in=given, final_state=True))
            return out + list(binding.ida_ssm_scan_backward(*args, dp, dy).values())
        work.append((call, [t.clone() for t in call()]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for k, (call, _) in enumerate(work):
            with torch.cuda.stream(streams[k]):
                got[k].append(call())
    _done()
    for k, (_, want) in enumerate(work):
        assert all(torch.equal(a, b) for out in got[k] for a, b in zip(out, want))


def test_gradients_of_no_positions_are_zero():
    for B, N in ((2, 0), (0, 5)):
        x = torch.empty(B, N, 3, 8, device="cuda", dtype=torch.bfloat16)
        bc = torch.empty(B, N, 1, 16, device="cuda", dtype=torch.bfloat16)
        g = binding.ida_ssm_scan_backward(x, bc, bc, x[..., 0], sc.cuda(sc.params(3, 8, 1, 1)), x)
        e, w = torch.empty(B, N, 16, device="cuda"), torch.ones(16, 4, device="cuda")
        h = binding.ida_ssm_conv_backward(e, e, w, w[:, 0].contiguous())
        _done()
        assert g["x"].numel() == 0 and h["x"].numel() == 0
        assert not any(t.any() for t in (g["a_log"], g["dt_bias"], g["D"], h["conv_w"], h["conv_b"]))


def _problem(dtype, B=3, N=1700, H=4, d=64, G=2, M=64):
    p, row, s, C = _scan_inputs(B, N, H, d, G, M, dtype, True, False)
    dy = torch.randn(B, N, H, d, generator=sc.gen(11)).to(sc.DT[dtype]).cuda()
    return (B, H, N, d, G, M), _on_gpu(row, C, H, d, G, M), sc.cuda(p), s.cuda(), dy


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_a_workspace_held_before_does_not_matter(dtype):
    """Results of split prompts and of gradients with workspaces full of NaN."""
    sizes, args, p, s, dy = _problem(dtype)
    code = binding.IDA_BF16 if dtype == "bf16" else binding.IDA_F32
    n = binding.ida_ssm_scan_workspace_bytes(*sizes, code), binding.ida_ssm_scan_backward_workspace_bytes(*sizes, code)
    full = [torch.full(((k + 3) // 4,), float("nan"), device="cuda") for k in n]
    assert n[0] > 0
    want = list(binding.ida_ssm_scan(*args, p, state_in=s, final_state=True))
    got = list(binding.ida_ssm_scan(*args, p, state_in=s, final_state=True, workspace=full[0]))
    full[0].fill_(float("nan"))
    got.append(binding.ida_ssm_scan(*args, p, state_in=s, workspace=full[0])[0])
    want.append(want[0])
    got += binding.ida_ssm_scan_backward(*args, p, dy, workspace=full[1]).values()
    want += binding.ida_ssm_scan_backward(*args, p, dy).values()
    x, w, b = dy.flatten(2), torch.ones(256, 4, device="cuda"), torch.ones(256, device="cuda")
    k = binding.ida_ssm_conv_backward_workspace_bytes(*x.shape, 4)
    got += binding.ida_ssm_conv_backward(x, x, w, b, workspace=torch.full((k // 4,), float("nan"), device="cuda")).values()
    want += binding.ida_ssm_conv_backward(x, x, w, b).values()
    k = binding.ida_rmsnorm_backward_workspace_bytes(x.shape[0] * x.shape[1], 256)
    got += binding.ida_rmsnorm_backward(x, b, x, workspace=torch.full((k // 4,), float("nan"), device="cuda")).values()
    want += binding.ida_rmsnorm_backward(x, b, x).values()
    _done()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_graphs_that_share_a_workspace(dtype):
    """A split prompt and gradients captured apart, over the same workspace, replayed in turn."""
    sizes, args, p, s, dy = _problem(dtype)
    code = binding.IDA_BF16 if dtype == "bf16" else binding.IDA_F32
    ws = torch.empty(max(binding.ida_ssm_scan_workspace_bytes(*sizes, code),
                         binding.ida_ssm_scan_backward_workspace_bytes(*sizes, code)), dtype=torch.uint8, device="cuda")
    calls = [lambda: list(binding.ida_ssm_scan(*args, p, state_in=s, final_state=True, workspace=ws)),
             lambda: list(binding.ida_ssm_scan_backward(*args, p, dy, workspace=ws).values())]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph, call in zip(graphs, calls):
        with torch.cuda.graph(graph):
            got.append(call())
    for _ in range(3):
        for outs in got:
            for t in outs:
                t.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        _done()
        assert all(torch.equal(a, c) for o, w in zip(got, want) for a, c in zip(o, w))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_rows_and_heads_than_a_grid_dimension(dtype):
    """68000 units of two positions: the sums over chunks take two launches."""
    case = (17000, 2, 4, 8, 2, 8, dtype, True, False)
    B, N, H, d, G, M = case[:6]
    p, row, s, C = _scan_inputs(*case)
    args, dp = _on_gpu(row, C, H, d, G, M), sc.cuda(p)
    y, X = binding.ida_ssm_scan(*args, dp, state_in=s.cuda(), final_state=True)
    dy = torch.randn(B, N, H, d, generator=sc.gen(11)).to(sc.DT[dtype])
    g = binding.ida_ssm_scan_backward(*args, dp, dy.cuda())
    _done()
    ry, rX = _scan_ref(row, C, H, d, G, M, p, s)
    ya, Xa = _scan_ref(row, C, H, d, G, M, p, s, absolute=True)
    by, bX = _scan_bounds(dtype, N, ry, ya, Xa)
    assert worst(y, ry, by) <= 1 and worst(X, rX, bX) <= 1
    # 17000 chunks (four parts each on the tensor cores) are added in 128 interleaved sums
    check_scan_gradients(g, row, C, H, d, G, M, p, dy, dtype, sums=4 * B // 128 + 8)
