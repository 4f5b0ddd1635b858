"""Pins of the oracle of the selective mixer and the pre-norm (oracle/ida_ssm.py): closed forms,
invariants and differences."""
import torch

from oracle import ida_ssm as orc
from tests.ssm_cases import params, split, to64


def _problem(B=2, N=13, H=4, d=3, G=2, M=5, W=4, seed=1):
    C = H * d + 2 * G * M
    g = torch.Generator().manual_seed(seed)
    xbc = torch.randn(B, N, C, generator=g, dtype=torch.float64)
    dt = torch.randn(B, N, H, generator=g, dtype=torch.float64)
    return xbc, dt, to64(params(H, C, W, seed)), (H, d, G, M)


def _scan(xbc, dt, p, shape, state=None):
    return orc.scan(*split(xbc, *shape), dt, p["a_log"], p["dt_bias"], p["D"], state)


def test_scan_is_the_decayed_sum_over_earlier_positions():
    """y_t = sum_{s<=t} exp(-rate (S_t - S_s)) D_s (c_t . b_s) x_s + D x_t with S the running sum of
    the step sizes."""
    xbc, dt, p, shape = _problem()
    y, _ = _scan(xbc, dt, p, shape)
    x, b, c = split(xbc, *shape)
    H, d, G, M = shape
    delta = orc.step_size(dt, p["dt_bias"])
    S = delta.cumsum(1)
    for h in range(H):
        g = h // (H // G)
        k = torch.einsum("btm,bsm->bts", c[:, :, g], b[:, :, g])
        k = k * torch.exp(-torch.exp(p["a_log"][h]) * (S[:, :, None, h] - S[:, None, :, h])) * delta[:, None, :, h]
        ref = k.tril() @ x[:, :, h] + p["D"][h] * x[:, :, h]
        assert torch.allclose(y[:, :, h], ref, rtol=1e-12, atol=1e-12)


def test_parts_of_a_prompt_and_single_positions_continue_it():
    xbc, dt, p, shape = _problem()
    H, d, G, M = shape
    act, tail = orc.conv(xbc, p["conv_w"], p["conv_b"])
    y, X = _scan(act, dt, p, shape)
    for cut in (1, 2, 6):
        a1, t1 = orc.conv(xbc[:, :cut], p["conv_w"], p["conv_b"])
        y1, X1 = _scan(a1, dt[:, :cut], p, shape)
        a2, t2 = orc.conv(xbc[:, cut:], p["conv_w"], p["conv_b"], t1)
        y2, X2 = _scan(a2, dt[:, cut:], p, shape, X1)
        assert torch.allclose(torch.cat([y1, y2], 1), y, rtol=1e-12, atol=1e-13)
        assert torch.allclose(X2, X, rtol=1e-12, atol=1e-13) and torch.equal(t2, tail)
        for t in range(cut, xbc.shape[1]):
            o, t1, X1 = orc.step(xbc[:, t], dt[:, t], p, t1, X1, G)
            assert torch.allclose(o, y[:, t], rtol=1e-12, atol=1e-13)


def test_conv_taps_and_rows():
    x = torch.tensor([[[1.0], [2.0], [4.0]]], dtype=torch.float64)
    out, tail = orc.conv(x, torch.tensor([[10.0, 1.0]], dtype=torch.float64), torch.tensor([0.5], dtype=torch.float64))
    pre = torch.tensor([1.5, 12.5, 24.5], dtype=torch.float64)  # 1, 2 + 10, 4 + 20
    assert torch.allclose(out[0, :, 0], pre * torch.sigmoid(pre), rtol=1e-14, atol=0)
    assert tail.tolist() == [[[4.0]]]


def test_step_size_at_both_ends():
    z = torch.tensor([-800.0, -30.0, 0.0, 30.0, 800.0], dtype=torch.float64)
    got = orc.step_size(z, torch.zeros(()))
    assert got[0] == 0.0 and abs(got[1] - torch.exp(z[1])) < 1e-25 and abs(got[2] - torch.log(torch.tensor(2.0).double())) < 1e-15
    assert torch.equal(got[4], z[4])


def test_gradients_agree_with_differences():
    xbc, dt, p, shape = _problem(B=1, N=5, H=2, d=2, G=1, M=3, W=3)
    g = torch.Generator().manual_seed(9)
    dy = torch.randn(1, 5, 2, 2, generator=g, dtype=torch.float64)
    x, b, c = (t.contiguous() for t in split(xbc, *shape))
    leaves = [x, b, c, dt, p["a_log"], p["dt_bias"], p["D"]]

    def fn(*v):
        return orc.scan(*v)[0]

    got = orc.grads(fn, leaves, dy)
    for k, leaf in enumerate(leaves):
        flat = leaf.reshape(-1)
        for i in range(flat.numel()):
            e = torch.zeros_like(flat)
            e[i] = 1e-5
            up = [v if j != k else (flat + e).reshape(leaf.shape) for j, v in enumerate(leaves)]
            dn = [v if j != k else (flat - e).reshape(leaf.shape) for j, v in enumerate(leaves)]
            diff = ((fn(*up) - fn(*dn)) * dy).sum() / 2e-5
            assert abs(diff - got[k].reshape(-1)[i]) <= 1e-8 * (1 + abs(diff))


def test_rmsnorm_of_a_constant_row_and_scale_invariance():
    w = torch.tensor([2.0, -1.0, 0.5], dtype=torch.float64)
    r = torch.full((1, 3), 7.0, dtype=torch.float64)
    assert torch.allclose(orc.rmsnorm(r, w, 0.0), w[None], rtol=1e-14, atol=0)
    r = torch.tensor([[1.0, -2.0, 3.0]], dtype=torch.float64)
    assert torch.allclose(orc.rmsnorm(r, w, 0.0), orc.rmsnorm(1e6 * r, w, 0.0), rtol=1e-13, atol=0)
