"""Gradients of the feed-forward block's weights over many rows, where a sum's own error counts."""
import pytest
import torch

from linear_token_mixer_sc_gb300 import binding
from tests.ssm_cases import DT

pytestmark = pytest.mark.gpu


def _case(T, D, F, dtype, seed=1):
    """Inputs of one sign, so that every product adds to its sum, in channels of unlike size, so that results lie anywhere
    between two neighbours of their type; and the weights' gradients in 64 bits."""
    g = torch.Generator("cuda").manual_seed(seed)

    def positive(rows, cols):
        size = torch.exp2(2 * torch.rand(cols, generator=g, device="cuda"))
        return ((0.5 + torch.rand(rows, cols, generator=g, device="cuda")) * size).to(DT[dtype])

    x, dy, wd = positive(T, D), positive(T, D), positive(D, F) / D
    wg, wu = torch.zeros(2, F, D, dtype=DT[dtype], device="cuda")  # (dx is not looked at)
    acts = torch.empty(3, T, F, dtype=DT[dtype], device="cuda")
    for a in acts:
        a.copy_(positive(T, F))
    want = {k: 0 for k in ("w_gate", "w_up", "w_down")}
    for r in range(0, T, 1 << 18):
        gate, up, h = acts[:, r:r + (1 << 18)].double().unbind()
        s, y, xr = torch.sigmoid(gate), dy[r:r + (1 << 18)].double(), x[r:r + (1 << 18)].double()
        dh = y @ wd.double()
        want["w_gate"] += (dh * up * s * (1 + gate * (1 - s))).t() @ xr
        want["w_up"] += (dh * gate * s).t() @ xr
        want["w_down"] += y.t() @ h
    return (x, wg, wu, wd, acts, dy), want


@pytest.mark.parametrize("T,D,F", [(1 << 20, 64, 64), (1 << 18, 1024, 1024), (70001, 200, 328)])
def test_bf16_sums_over_many_rows(T, D, F):
    """Sums keep their size however many rows they have.  Tensor cores cut a running sum off by less than 2^-23 of it
    every 16 rows: of 4096 rows by less than 2^-15, and the sums of 4096 rows each are added in fp32, at most
    2^-24 of the whole each, 2^-16 for 2^20 rows.  The results' own roundings, 2^-8 each at most, are of either sign:
    their mean over at least 4096 results is below 6 / sqrt(3 * 4096) 2^-9 (the least step's half is 2^-9 of the value),
    about 2^-13; so are those of dg and du, over the rows as well."""
    args, want = _case(T, D, F, "bf16")
    got = binding.ida_ffn_backward(*args)
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
    for k, v in want.items():
        rel = got[k].double() / v - 1
        assert abs(float(rel.mean())) <= 2.0 ** -12, k
        # dg and du are rounded too, each 2^-8 at most; w_down's inputs are given
        assert float(rel.abs().max()) <= 2.0 ** -8 * (1 if k == "w_down" else 2) + 2.0 ** -14, k


@pytest.mark.parametrize("T,D,F", [(1 << 21, 8, 8), (65536, 32, 64), (20003, 72, 136), (1500, 40, 24), (1024, 16, 8), (300000, 128, 128), (30000, 128, 136)])
def test_fp32_sums_over_many_rows(T, D, F):
    """Weights' gradients of many rows and few channels, in a workspace of NaN and of no more bytes than asked for.
    On the CUDA cores a thread's sum has a quarter of a part's rows, of at most 1024 rows or a share of them that takes
    608 blocks; each addition is off by at most 2^-24 of the sum, and all terms have one sign.  dh is a sum of D
    products; sigmoid and the products behind it are off by less than 2^-19.  On the tensor cores (the last case) 512 rows
    are summed at a time, below 2^-18 in 32 steps with their alignments, and those sums in fp32, six times over."""
    args, want = _case(T, D, F, "f32")
    n = binding.ida_ffn_backward_workspace_bytes(T, D, F, 0)
    raw = torch.full((n + 131072,), 255, dtype=torch.uint8, device="cuda")
    got = binding.ida_ffn_backward(*args, workspace=raw[65536:65536 + n])
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
    assert bool((raw[:65536] == 255).all()) and bool((raw[65536 + n:] == 255).all())
    tiles = 3 * -(-D // 32) * -(-F // 32)
    terms = max(1024, -(-T * tiles // 608) + 64) / 4 + 608 + D if D * F <= 1 << 14 or T * D * F <= 1 << 27 else T / 512 * 6 + 64
    for k, v in want.items():
        rel = (got[k].double() / v - 1).abs()
        assert float(rel.max()) <= terms * 2.0 ** -24 + 2.0 ** -18, k


def test_fp32_gradients_of_few_channels_share_their_rows():
    """2^21 rows of 8 channels (some 0.4 GB to read and write, 1.4 ms): not three blocks that walk all rows (24 ms)."""
    args, _ = _case(1 << 21, 8, 8, "f32")
    binding.ida_ffn_backward(*args)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    binding.ida_ffn_backward(*args)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) <= 8


@pytest.mark.parametrize("dtype,T,D,F", [("f32", 20003, 72, 136), ("bf16", 70001, 40, 72)])
def test_captured_and_on_another_stream(dtype, T, D, F):
    args, _ = _case(T, D, F, dtype)
    want = {k: t.clone() for k, t in binding.ida_ffn_backward(*args).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = binding.ida_ffn_backward(*args)
    side.synchronize()
    assert all(torch.equal(got[k], w) for k, w in want.items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.ida_ffn_backward(*args)
        again = binding.ida_ffn_backward(*args)
    for _ in range(3):
        for t in (*got.values(), *again.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], w) and torch.equal(again[k], w) for k, w in want.items())
