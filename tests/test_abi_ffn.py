"""Refusals of the feed-forward block's and the 8-bit products' entry points: through the C ABI with addresses that
are never dereferenced, and through the binding."""
import ctypes

import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build

# a call that were not refused would run on addresses that are made up
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a CUDA device")

ARG, UNS, OK, CUDA = binding.IDA_ERR_ARG, binding.IDA_ERR_UNSUPPORTED, binding.IDA_OK, binding.IDA_ERR_CUDA
T, D, F = 300, 256, 384
X, DF, TF = 2 * T * D, 2 * D * F, 2 * T * F
KB, FB = D // 128, F // 128
FEW = 6  # rows of the block's call: of few, the workspace is needed beside acts
FX, FTF = 2 * FEW * D, 2 * FEW * F


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


# call: (arguments in their order, {output: bytes}, {input: bytes}, the rest by name)
CALLS = {
    "ida_ffn": ("x wg wu wd out acts", dict(out=FX, acts=3 * FTF, ws=None), dict(x=FX, wg=DF, wu=DF, wd=DF),
                dict(rows=FEW, D=D, F=F, ldx=D, dtype=1, ws="ws", n=1 << 40, stream=None)),
    "ida_ffn_backward": ("x wg wu wd acts dout dx dwg dwu dwd", dict(dx=X, dwg=DF, dwu=DF, dwd=DF, ws=None),
                         dict(x=X, wg=DF, wu=DF, wd=DF, acts=3 * TF, dout=X),
                         dict(rows=T, D=D, F=F, ldx=D, dtype=1, ws="ws", n=1 << 40, stream=None)),
    "ida_quant_e4m3": ("x q s", dict(q=T * D, s=4 * T * KB), dict(x=X), dict(rows=T, K=D, block=1, ldx=D, dtype=1, stream=None)),
    "ida_gemm_e4m3": ("a sa b sb out", dict(out=2 * T * F), dict(a=T * D, sa=4 * T * KB, b=F * D, sb=4 * FB * KB),
                      dict(rows=T, K=D, N=F, dtype=1, stream=None)),
    "ida_glu_e4m3": ("a sa wg sg wu su q s", dict(q=T * F, s=4 * T * FB),
                     dict(a=T * D, sa=4 * T * KB, wg=F * D, sg=4 * FB * KB, wu=F * D, su=4 * FB * KB),
                     dict(rows=T, D=D, F=F, stream=None)),
}


def _sizes(name):
    outs = dict(CALLS[name][1])
    if "ws" in outs:
        outs["ws"] = (binding.ida_ffn_workspace_bytes(FEW, D, F, 1, True) if name == "ida_ffn" else
                      binding.ida_ffn_backward_workspace_bytes(T, D, F, 1))
    return outs, CALLS[name][2]


def _apart(name):
    outs, ins = _sizes(name)
    return {k: (1 << 40) + (i << 26) for i, k in enumerate([*outs, *ins])}


def _call(lib, name, at, **over):
    order, _, _, rest = CALLS[name]
    rest = {**rest, **over}
    ptr = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731
    return getattr(lib, name)(*[ptr(at[k]) for k in order.split()], *[ptr(at["ws"]) if v == "ws" else v for v in rest.values()])


BAD = {
    "ida_ffn": [(dict(rows=-1), ARG), (dict(D=0), ARG), (dict(F=0), ARG), (dict(D=252), UNS), (dict(F=388), UNS), (dict(D=65544, ldx=65544), UNS),
                (dict(F=65544), UNS), (dict(dtype=2), ARG), (dict(ldx=248), ARG), (dict(ldx=260), UNS), (dict(ldx=(1 << 32) + 8), UNS),
                (dict(rows=(1 << 28) + 1), UNS), (dict(rows=1 << 27, F=1024), UNS), (dict(n=16), ARG)],
    "ida_quant_e4m3": [(dict(rows=-1), ARG), (dict(K=0), ARG), (dict(K=248), UNS), (dict(K=65552, ldx=65552), UNS), (dict(block=2), UNS),
                       (dict(dtype=-1), ARG), (dict(ldx=240), ARG), (dict(ldx=260), UNS), (dict(rows=(1 << 28) + 1), UNS)],
    "ida_gemm_e4m3": [(dict(rows=-1), ARG), (dict(K=0), ARG), (dict(N=0), ARG), (dict(K=264), UNS), (dict(N=12), UNS), (dict(dtype=3), ARG),
                      (dict(K=65552), UNS), (dict(N=65544), UNS), (dict(rows=1 << 28, N=512), UNS)],
    "ida_glu_e4m3": [(dict(rows=-1), ARG), (dict(D=0), ARG), (dict(F=0), ARG), (dict(D=264), UNS), (dict(F=392), UNS), (dict(F=65552), UNS)],
}
BAD["ida_ffn_backward"] = BAD["ida_ffn"]


@no_device
@pytest.mark.parametrize("name", CALLS)
def test_sizes_and_pointers(lib, name):
    at = _apart(name)
    for over, want in BAD[name]:
        assert _call(lib, name, at, **over) == want, over
    for k in CALLS[name][0].split():
        if (name, k) != ("ida_ffn", "acts"):
            assert _call(lib, name, {**at, k: None}) == ARG, k
        for off in (1, 4, 8):
            assert _call(lib, name, {**at, k: at[k] + off}) == ARG and "aligned" in binding.ida_last_error(), (k, off)
    if name == "ida_ffn":  # more rows need none beside acts
        assert _call(lib, name, {**at, "ws": None}, rows=T, n=0) == CUDA
        assert _call(lib, name, {**at, "ws": None, "acts": None}, rows=T, n=0) == ARG
    if "ws" in at:
        assert _call(lib, name, {**at, "ws": None}) == ARG and _call(lib, name, {**at, "ws": at["ws"] + 4}) == ARG
    assert _call(lib, name, at) == CUDA  # nothing else is wrong with it


@no_device
@pytest.mark.parametrize("name", CALLS)
def test_every_output_over_every_other_tensor(lib, name):
    outs, ins = _sizes(name)
    sizes = {**outs, **ins}
    for o in outs:
        for k in sizes:
            if k != o:
                base = _apart(name)
                for at in {base[k] + (sizes[k] - 1) // 16 * 16, base[k] - (sizes[o] - 1) // 16 * 16, base[k]}:
                    assert _call(lib, name, {**base, o: at}) == ARG and "overlap" in binding.ida_last_error(), (o, k)
    base, at = {}, 1 << 40
    for k in sizes:
        base[k], at = at, at + (sizes[k] + 15) // 16 * 16
    assert _call(lib, name, base) == CUDA  # side by side


@no_device
def test_no_rows(lib):
    none = lambda name: {k: None for k in _apart(name)}  # noqa: E731
    for name in ("ida_ffn", "ida_quant_e4m3", "ida_gemm_e4m3", "ida_glu_e4m3"):
        assert _call(lib, name, none(name), rows=0) == OK
    assert _call(lib, "ida_ffn_backward", none("ida_ffn_backward"), rows=0) == ARG  # the weights' gradients are written
    back = {**none("ida_ffn_backward"), **{k: v for k, v in _apart("ida_ffn_backward").items() if k in ("dwg", "dwu", "dwd", "wg", "wu", "wd")}}
    assert _call(lib, "ida_ffn_backward", back, rows=0) == CUDA
    assert _call(lib, "ida_ffn_backward", {**back, "dwg": back["dwu"] + 16}, rows=0) == ARG


def test_workspaces(lib):
    keep = binding.ida_ffn_workspace_bytes
    assert keep(300, 256, 384, 1, True) == 0 and keep(300, 256, 384, 0, True) == 0  # acts take the hidden product
    assert keep(5, 256, 384, 1, True) > 0 and keep(5000, 256, 384, 0, True) > 0  # in two parts; fp32's parts
    for fn in (binding.ida_ffn_workspace_bytes, binding.ida_ffn_backward_workspace_bytes):
        for bad in [(0, 64, 64, 1), (-1, 64, 64, 1), (5, 60, 64, 1), (5, 64, 0, 1), (5, 64, 64, 2), (5, 65544, 64, 1)]:
            assert fn(*bad) == 0
        assert 0 < fn(7, 64, 64, 1) <= fn(7, 64, 64, 0) < fn(700, 64, 64, 0) < fn(70000, 64, 64, 0)
        with pytest.raises(ValueError, match="2\\^31"):
            fn(1 << 31, 64, 64, 1)
    assert keep(1, 2048, 5632, 0) < 1 << 20  # no parts of weights where no product takes them
    assert binding.ida_ffn_workspace_bytes(300, 256, 384, 1) >= 300 * 384 * 2


def test_host_tensors_and_names(lib):
    x, w, d = torch.zeros(4, 16), torch.zeros(32, 16), torch.zeros(16, 32)
    q, s, b = (torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.zeros(4, 1), torch.zeros(32, 16).to(torch.float8_e4m3fn))
    sb = torch.zeros(1, 1)
    for fn, kw in [(binding.ida_ffn, dict(x=x, w_gate=w, w_up=w, w_down=d)),
                   (binding.ida_ffn_backward, dict(x=x, w_gate=w, w_up=w, w_down=d, acts=torch.zeros(3, 4, 32), dout=x)),
                   (binding.ida_quant_e4m3, dict(x=x)), (binding.ida_gemm_e4m3, dict(a=q, a_scale=s, b=b, b_scale=sb)),
                   (binding.ida_glu_e4m3, dict(a=q, a_scale=s, w_gate=b, gate_scale=sb, w_up=b, up_scale=sb))]:
        with pytest.raises(ValueError, match="CUDA"):
            fn(**kw)
        with pytest.raises(TypeError, match=next(iter(kw))):
            fn()


@pytest.mark.gpu
def test_shapes_types_and_devices(lib):
    f = dict(device="cuda")
    x, wg, wd = torch.zeros(4, 16, **f), torch.zeros(32, 16, **f), torch.zeros(16, 32, **f)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        binding.ida_ffn(x.half(), wg.half(), wg.half(), wd.half())
    with pytest.raises(TypeError, match="w_up"):
        binding.ida_ffn(x, wg, wg.bfloat16(), wd)
    with pytest.raises(ValueError, match="w_down"):
        binding.ida_ffn(x, wg, wg, wg)
    with pytest.raises(ValueError, match="16 channels"):
        binding.ida_ffn(torch.zeros(4, 24, **f), wg, wg, wd)
    with pytest.raises(ValueError, match="w_gate"):
        binding.ida_ffn(x, torch.zeros(16, 32, **f).t(), wg, wd)
    with pytest.raises(ValueError, match="rows of x"):
        binding.ida_ffn(torch.zeros(4, 32, **f)[:, ::2], wg, wg, wd)
    with pytest.raises(ValueError, match="acts"):
        binding.ida_ffn(x, wg, wg, wd, acts=torch.zeros(2, 4, 32, **f))
    with pytest.raises(binding.IdaError, match="workspace"):
        binding.ida_ffn(x, wg, wg, wd, workspace=torch.zeros(16, **f))
    with pytest.raises(ValueError, match="acts"):
        binding.ida_ffn_backward(x, wg, wg, wd, torch.zeros(3, 5, 32, **f), x)
    q, s = binding.ida_quant_e4m3(x)
    qw, sw = binding.ida_quant_e4m3(wg, rows=128)
    with pytest.raises(binding.IdaError, match="block_rows"):
        binding.ida_quant_e4m3(x, rows=64)
    with pytest.raises(ValueError, match=r"\[N, K\]"):
        binding.ida_quant_e4m3(x[None], rows=128)
    with pytest.raises(TypeError, match="b must be"):
        binding.ida_gemm_e4m3(q, s, wg, sw)
    with pytest.raises(ValueError, match="a_scale"):
        binding.ida_gemm_e4m3(q, s[:2], qw, sw)
    with pytest.raises(ValueError, match="b_scale"):
        binding.ida_gemm_e4m3(q, s, qw, torch.zeros(2, 1, **f))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        binding.ida_gemm_e4m3(q, s, qw, sw, dtype=torch.float16)
    with pytest.raises(ValueError, match="w_up"):
        binding.ida_glu_e4m3(q, s, qw, sw, qw[:16], sw)
