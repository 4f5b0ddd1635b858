"""Outputs over inputs or one another are refused by every call of the selective mixer and of the
pre-norm, through the C ABI with addresses that are never dereferenced."""
import ctypes

import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build

# a call that were not refused would run on addresses that are made up
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a CUDA device")

ARG = binding.IDA_ERR_ARG
F = ctypes.c_float
B, N, H, d, G, M, W = 2, 5, 4, 64, 2, 16, 4
C = H * d + 2 * G * M
XBC = 2 * B * N * C


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _par(*names):
    return {k: 4 * H for k in names}


# call: (arguments in their order, {output: bytes}, {input: bytes}, pairs that may be the same tensor)
CALLS = {
    "ida_ssm_conv": ("x w bias si out fs", dict(out=XBC, fs=4 * B * (W - 1) * C),
                     dict(x=XBC, w=4 * C * W, bias=4 * C, si=4 * B * (W - 1) * C), (B, N, C, C, 1, W, None), ()),
    "ida_ssm_conv_backward": ("x dout w bias dx dw db", dict(dx=XBC, dw=4 * C * W, db=4 * C, ws=None),
                              dict(x=XBC, dout=XBC, w=4 * C * W, bias=4 * C), (B, N, C, C, C, 1, W, "ws", 1 << 30, None), ()),
    "ida_ssm_scan": ("x b c dt a bias D si y fs", dict(y=2 * B * N * H * d, fs=4 * B * H * M * d),
                     dict(x=2 * B * N * H * d, b=2 * B * N * G * M, c=2 * B * N * G * M, dt=2 * B * N * H,
                          si=4 * B * H * M * d, **_par("a", "bias", "D")),
                     (B, H, N, d, G, M, H * d, G * M, G * M, H, 1, None, 0, None), ()),
    "ida_ssm_scan_backward": ("x b c dt a bias D dy dx db dc ddt da dbias dD",
                              dict(dx=2 * B * N * H * d, db=2 * B * N * G * M, dc=2 * B * N * G * M, ddt=2 * B * N * H,
                                   ws=None, **_par("da", "dbias", "dD")),
                              dict(x=2 * B * N * H * d, b=2 * B * N * G * M, c=2 * B * N * G * M, dt=2 * B * N * H,
                                   dy=2 * B * N * H * d, **_par("a", "bias", "D")),
                              (B, H, N, d, G, M, H * d, G * M, G * M, H, H * d, G * M, G * M, H, 1, "ws", 1 << 40, None), ()),
    "ida_ssm_step": ("x dt w cb a bias D tail X y", dict(tail=4 * B * (W - 1) * C, X=4 * B * H * M * d, y=2 * B * H * d),
                     dict(x=2 * B * C, dt=2 * B * H, w=4 * C * W, cb=4 * C, **_par("a", "bias", "D")),
                     (B, H, d, G, M, C, H, 1, W, None), ()),
    "ida_rmsnorm": ("x res w ro out q sc", dict(ro=2 * 9 * 256, out=2 * 9 * 256, q=9 * 256, sc=4 * 9 * 4),
                    dict(x=2 * 9 * 256, res=2 * 9 * 256, w=4 * 256), (9, 256, 64, F(1e-6), 1, None),
                    (("ro", "x"), ("ro", "res"))),
    "ida_rmsnorm_backward": ("r w dy dres dx dw", dict(dx=2 * 9 * 256, dw=4 * 256, ws=None),
                             dict(r=2 * 9 * 256, w=4 * 256, dy=2 * 9 * 256, dres=2 * 9 * 256),
                             (9, 256, F(1e-6), 1, "ws", 1 << 30, None), (("dx", "dy"), ("dx", "dres"))),
}


def _outputs(name):
    """The outputs' bytes, with the workspace's as the library states them."""
    outs = dict(CALLS[name][1])
    if "ws" in outs:
        outs["ws"] = {"ida_ssm_conv_backward": lambda: binding.ida_ssm_conv_backward_workspace_bytes(B, N, C, W),
                      "ida_ssm_scan_backward": lambda: binding.ida_ssm_scan_backward_workspace_bytes(B, H, N, d, G, M, 1),
                      "ida_rmsnorm_backward": lambda: binding.ida_rmsnorm_backward_workspace_bytes(9, 256)}[name]()
    return outs


def _call(lib, name, at):
    order, _, _, rest, _ = CALLS[name]
    args = [ctypes.c_void_p(at[k]) for k in order.split()]
    return getattr(lib, name)(*args, *(ctypes.c_void_p(at["ws"]) if r == "ws" else r for r in rest))


def _apart(name):
    outs, ins = _outputs(name), CALLS[name][2]
    return {k: (1 << 40) + (i << 24) for i, k in enumerate([*outs, *ins])}


@pytest.mark.parametrize("name", CALLS)
def test_every_output_over_every_other_tensor(lib, name):
    """From behind and from before, by 16 bytes; the same tensor, where it may not be that."""
    outs, ins, same = _outputs(name), CALLS[name][2], CALLS[name][4]
    sizes = {**outs, **ins}
    for o in outs:
        for k in sizes:
            if k == o:
                continue
            base = _apart(name)
            ends = {base[k] + (sizes[k] - 1) // 16 * 16, base[k] - (sizes[o] - 1) // 16 * 16, base[k]}
            for at in sorted(ends - ({base[k]} if (o, k) in same else set())):
                got = _call(lib, name, {**base, o: at})
                assert got == ARG and "overlap" in binding.ida_last_error(), (o, k, at - base[k])


@pytest.mark.parametrize("name", CALLS)
def test_tensors_side_by_side_are_taken(lib, name):
    """Nothing is refused for its place (what stops these calls is that there is no device)."""
    outs, ins, same = _outputs(name), CALLS[name][2], CALLS[name][4]
    sizes = {**outs, **ins}
    base, at = {}, 1 << 40
    for k in sizes:
        base[k], at = at, at + (sizes[k] + 15) // 16 * 16
    for pair in (None, *same):
        here = dict(base) if pair is None else {**base, pair[0]: base[pair[1]]}
        assert _call(lib, name, here) == binding.IDA_ERR_CUDA, pair


def test_gradient_rows_of_other_strides_and_slices_of_the_same_rows(lib):
    """dx in the same wider rows as x is taken where it is another slice of them, and refused at another
    stride."""
    base = _apart("ida_ssm_conv_backward")
    order = CALLS["ida_ssm_conv_backward"][0].split()

    def call(dx, ldx, lddx):
        at = {**base, "dx": dx}
        args = [ctypes.c_void_p(at[k]) for k in order]
        return lib.ida_ssm_conv_backward(*args, B, N, C, ldx, lddx, 1, W, ctypes.c_void_p(at["ws"]), 1 << 30, None)

    for off in (0, 2 * C - 16, 2 * (2 * C) - 16):
        assert call(base["x"] + off, 2 * C, 2 * C) == ARG and "overlap" in binding.ida_last_error(), off
    assert call(base["x"] + 2 * C, 2 * C, 3 * C) == ARG and "overlap" in binding.ida_last_error()
    assert call(base["x"] + 2 * C, 2 * C, 2 * C) == binding.IDA_ERR_CUDA
