"""Refusals of the selective mixer's and the pre-norm's entry points: through the C ABI with host
addresses standing in for device ones (every call here is refused, or has nothing to do, before
the library touches CUDA), and through the binding."""
import ctypes

import pytest
import torch

from linear_token_mixer_sc_gb300 import binding, build
from tests.test_abi_host import _Bufs

ARG, UNS, OK = binding.IDA_ERR_ARG, binding.IDA_ERR_UNSUPPORTED, binding.IDA_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _caller(fn, names, defaults):
    def call(**over):
        kw = dict(defaults, **over)
        return fn(*[kw[n] for n in names])
    return call


def _conv(lib, b):
    names = "x w bias si out fs B N C ldx dtype W stream".split()
    return _caller(lib.ida_ssm_conv, names, dict(x=b.p, w=b.p, bias=b.p, si=None, out=b.p, fs=None, B=2, N=5, C=32,
                                                 ldx=32, dtype=1, W=4, stream=None))


def _scan(lib, b):
    names = "x b c dt a bias D si y fs B H N d G M ldx ldb ldc lddt dtype ws n stream".split()
    return _caller(lib.ida_ssm_scan, names,
                   dict(x=b.p, b=b.p, c=b.p, dt=b.p, a=b.p, bias=b.p, D=b.p, si=None, y=b.p, fs=None, B=1, H=4, N=9,
                        d=64, G=2, M=16, ldx=256, ldb=32, ldc=32, lddt=4, dtype=1, ws=None, n=0, stream=None))


SCAN_BAD = [(dict(d=12), UNS), (dict(d=264, ldx=1056), UNS), (dict(M=136, ldb=272, ldc=272), UNS), (dict(M=4), UNS),
            (dict(G=3), ARG), (dict(G=0), ARG), (dict(B=-1), ARG), (dict(N=-1), ARG), (dict(dtype=2), ARG),
            (dict(ldx=248), ARG), (dict(ldx=260), UNS), (dict(ldb=36), UNS), (dict(ldb=24), ARG), (dict(ldc=36), UNS), (dict(ldc=24), ARG), (dict(lddt=3), ARG),
            (dict(B=1 << 23), UNS), (dict(N=(1 << 28) + 1), UNS), (dict(ldx=(1 << 32) + 8), UNS)]


def test_scan_refusals(lib):
    b = _Bufs()
    call = _scan(lib, b)
    for over, want in SCAN_BAD:
        assert call(**over) == want, over
    for k in ("x", "b", "c", "dt", "a", "bias", "D", "y"):
        assert call(**{k: None}) == ARG, k
    for k in ("x", "b", "c", "a", "bias", "D", "y", "si", "fs", "ws"):
        assert call(**{k: b.mis}) == ARG, k
    assert call(dt=ctypes.c_void_p(b.p.value + 1)) == ARG
    assert call(si=b.p, fs=b.p) == ARG and "overlap" in binding.ida_last_error()
    assert call(si=b.p, fs=ctypes.c_void_p(b.p.value + 64)) == ARG
    assert call(B=0, x=None) == OK and call(H=0, ldx=0, lddt=0) == OK and call(N=0, x=None, y=None) == OK


def test_conv_refusals(lib):
    b = _Bufs()
    call = _conv(lib, b)
    for over, want in [(dict(B=-1), ARG), (dict(N=-2), ARG), (dict(C=0), ARG), (dict(C=20), UNS), (dict(W=0), ARG),
                       (dict(W=5), UNS), (dict(dtype=5), ARG), (dict(ldx=24), ARG), (dict(ldx=36), UNS),
                       (dict(C=(1 << 20) + 8, ldx=1 << 21), UNS), (dict(N=1 << 28), UNS)]:
        assert call(**over) == want, over
    for k in ("x", "w", "bias", "out"):
        assert call(**{k: None}) == ARG and call(**{k: b.mis}) == ARG, k
    assert call(si=b.mis) == ARG and call(fs=b.mis) == ARG and call(si=b.p, fs=b.p) == ARG
    assert call(B=0, x=None) == OK and call(N=0, x=None) == OK
    names = "x dout w bias dx dw db B N C ldx lddx dtype W ws n stream".split()
    back = _caller(lib.ida_ssm_conv_backward, names, dict(x=b.p, dout=b.p, w=b.p, bias=b.p, dx=b.p, dw=b.p, db=b.p,
                                                          B=2, N=5, C=32, ldx=32, lddx=32, dtype=1, W=4, ws=b.p,
                                                          n=1 << 30, stream=None))
    for k in ("x", "dout", "w", "bias", "dx", "dw", "db", "ws"):
        assert back(**{k: None}) == ARG, k
    assert back(n=16) == ARG and "workspace" in binding.ida_last_error()
    assert back(lddx=36) == UNS and back(lddx=16) == ARG and back(W=6) == UNS
    assert binding.ida_ssm_conv_backward_workspace_bytes(2, 5, 32, 4) > 0
    for bad in ((0, 5, 32, 4), (2, 0, 32, 4), (2, 5, 30, 4), (2, 5, 32, 5)):
        assert binding.ida_ssm_conv_backward_workspace_bytes(*bad) == 0


def test_scan_backward_refusals(lib):
    b = _Bufs()
    names = ("x b c dt a bias D dy dx db dc ddt da dbias dD B H N d G M ldx ldb ldc lddt lddx lddb lddc ldddt dtype ws n "
             "stream").split()
    ptrs = names[:15]
    call = _caller(lib.ida_ssm_scan_backward, names,
                   dict({k: b.p for k in ptrs}, B=1, H=4, N=9, d=64, G=2, M=16, ldx=256, ldb=32, ldc=32, lddt=4, lddx=256,
                        lddb=32, lddc=32, ldddt=4, dtype=1, ws=b.p, n=1 << 40, stream=None))
    for k in ptrs + ["ws"]:
        assert call(**{k: None}) == ARG, k
    for over, want in SCAN_BAD + [(dict(lddx=248), ARG), (dict(lddx=260), UNS), (dict(lddb=36), UNS), (dict(lddc=24), ARG),
                                  (dict(ldddt=2), ARG), (dict(n=1024), ARG)]:
        assert call(**over) == want, over
    assert call(H=0, ldx=0, lddt=0, lddx=0, ldddt=0) == OK
    n = binding.ida_ssm_scan_backward_workspace_bytes(1, 4, 9, 64, 2, 16, 1)
    assert n > 0 and n % 16 == 0
    assert binding.ida_ssm_scan_backward_workspace_bytes(1, 4, 0, 64, 2, 16, 1) == 0
    assert binding.ida_ssm_scan_backward_workspace_bytes(1, 4, 9, 60, 2, 16, 1) == 0
    if not torch.cuda.is_available():
        assert binding.ida_ssm_scan_workspace_bytes(1, 4, 4096, 64, 2, 16, 1) == 0


def test_outputs_over_inputs_are_refused(lib):
    b = _Bufs()
    at = lambda off: ctypes.c_void_p(b.p.value + off)
    assert _conv(lib, b)() == ARG and "overlap" in binding.ida_last_error()
    assert _conv(lib, b)(out=at(2 * 32 * 9)) == ARG  # x's last row
    for off in (0, 2 * 256 * 8, 2 * 256 * 9 - 16):
        assert _scan(lib, b)(y=at(off)) == ARG and "overlap" in binding.ida_last_error(), off
    far = at(1 << 24)
    assert _scan(lib, b)(x=far, y=at(-2 * 256 * 8)) == ARG and "overlap" in binding.ida_last_error()  # y's last row on b, c, dt
    names = "x dout w bias dx dw db B N C ldx lddx dtype W ws n stream".split()
    back = _caller(lib.ida_ssm_conv_backward, names, dict(x=b.p, dout=far, w=b.p, bias=b.p, dx=b.p, dw=b.p, db=b.p,
                                                          B=2, N=5, C=32, ldx=96, lddx=96, dtype=1, W=4, ws=b.p,
                                                          n=1 << 30, stream=None))
    for kw in (dict(), dict(dx=far), dict(dx=at(48)), dict(dx=at(2 * 80)), dict(dx=at(2 * 48), lddx=64)):
        assert back(**kw) == ARG and "overlap" in binding.ida_last_error(), kw


def test_step_refusals(lib):
    b = _Bufs()
    names = "xbc dt w cb a bias D tail X y B H d G M ldx lddt dtype W stream".split()
    call = _caller(lib.ida_ssm_step, names, dict(xbc=b.p, dt=b.p, w=b.p, cb=b.p, a=b.p, bias=b.p, D=b.p, tail=b.p,
                                                 X=b.p, y=b.p, B=1, H=4, d=64, G=2, M=16, ldx=320, lddt=4, dtype=1,
                                                 W=4, stream=None))
    for over, want in [(dict(B=-1), ARG), (dict(H=-4), ARG), (dict(W=0), ARG), (dict(W=5), UNS), (dict(d=20), UNS),
                       (dict(M=136), UNS), (dict(G=3), ARG), (dict(ldx=312), ARG), (dict(ldx=324), UNS),
                       (dict(lddt=2), ARG), (dict(dtype=9), ARG), (dict(B=1 << 27), UNS)]:
        assert call(**over) == want, over
    for k in ("xbc", "dt", "w", "cb", "a", "bias", "D", "tail", "X", "y"):
        assert call(**{k: None}) == ARG, k
        if k != "dt":
            assert call(**{k: b.mis}) == ARG, k
    assert call(B=0, xbc=None) == OK


def test_norm_refusals(lib):
    b = _Bufs()
    F = ctypes.c_float
    names = "x res w ro out q sc rows D group eps dtype stream".split()
    call = _caller(lib.ida_rmsnorm, names, dict(x=b.p, res=None, w=b.p, ro=None, out=b.p, q=b.p, sc=b.p, rows=3, D=256,
                                                group=0, eps=F(1e-6), dtype=1, stream=None))
    for over, want in [(dict(rows=-1), ARG), (dict(D=4), UNS), (dict(D=12), UNS), (dict(D=8200), UNS),
                       (dict(group=-1), ARG), (dict(group=48), UNS), (dict(group=128, D=192), UNS), (dict(dtype=3), ARG),
                       (dict(eps=F(-1.0)), ARG), (dict(eps=F(float("nan"))), ARG), (dict(eps=F(float("inf"))), ARG),
                       (dict(x=None), ARG), (dict(w=None), ARG), (dict(out=None), ARG), (dict(group=64, q=None), ARG),
                       (dict(group=64, sc=None), ARG), (dict(res=b.mis), ARG), (dict(ro=b.mis), ARG), (dict(x=b.mis), ARG)]:
        assert call(**over) == want, over
    assert call(rows=0, x=None) == OK
    names = "r w dy dres dx dw rows D eps dtype ws n stream".split()
    back = _caller(lib.ida_rmsnorm_backward, names, dict(r=b.p, w=b.p, dy=b.p, dres=None, dx=b.p, dw=b.p, rows=3, D=256,
                                                         eps=F(1e-6), dtype=1, ws=b.p, n=1 << 30, stream=None))
    for k in ("r", "w", "dy", "dx", "dw", "ws"):
        assert back(**{k: None}) == ARG and back(**{k: b.mis}) == ARG, k
    assert back(n=64) == ARG and back(D=8200) == UNS and back(dres=b.mis) == ARG
    assert binding.ida_rmsnorm_backward_workspace_bytes(0, 256) == 0
    assert binding.ida_rmsnorm_backward_workspace_bytes(3, 256) >= 256 * 4


def test_binding_refuses_host_tensors(lib):
    t = torch.zeros(1, 8, 16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.ida_ssm_conv(t, t[0, :, :4], t[0, 0])
    with pytest.raises(ValueError, match="CUDA"):
        binding.ida_rmsnorm(t, t[0, 0])


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit(lib):
    f = dict(device="cuda")
    x, w = torch.zeros(2, 9, 64, **f), torch.zeros(64, 4, **f)
    b = w[:, 0].contiguous()
    with pytest.raises(ValueError, match="dense"):
        binding.ida_ssm_conv(torch.zeros(2, 9, 128, **f)[..., ::2], w, b)
    with pytest.raises(ValueError, match="one stride"):
        binding.ida_ssm_conv(torch.zeros(2, 12, 64, **f)[:, :9], w, b)
    with pytest.raises(ValueError, match="shape"):
        binding.ida_ssm_conv(x, torch.zeros(60, 4, **f), b)
    with pytest.raises(TypeError, match="float32"):
        binding.ida_ssm_conv(x, w.bfloat16(), b)
    with pytest.raises(TypeError):
        binding.ida_ssm_conv(x.half(), w, b)
    with pytest.raises(binding.IdaError, match="row stride"):
        binding.ida_ssm_conv(torch.zeros(2, 1, 64, **f).expand(2, 9, 64)[:1], w, b)
    p = {k: torch.zeros(2, **f) for k in ("a_log", "dt_bias", "D")}
    xs, bc, dt = torch.zeros(1, 9, 2, 32, **f), torch.zeros(1, 9, 1, 16, **f), torch.zeros(1, 9, 2, **f)
    with pytest.raises(ValueError, match="shape"):
        binding.ida_ssm_scan(xs, bc, bc[:, :8], dt, p)
    with pytest.raises(binding.IdaError, match="strides"):
        binding.ida_ssm_scan(xs, bc, torch.zeros(1, 9, 1, 20, **f)[..., :16], dt, p)
    with pytest.raises(TypeError):
        binding.ida_ssm_scan(xs, bc, bc, dt.bfloat16(), p)
    with pytest.raises(ValueError, match="final_state"):
        binding.ida_ssm_scan(xs, bc, bc, dt, p, final_state=torch.zeros(1, 2, 32, 16, **f))
    with pytest.raises(ValueError, match="channels"):
        binding.ida_ssm_step(torch.zeros(1, 90, **f), dt[:, 0], {**p, "conv_w": w, "conv_b": b},
                             torch.zeros(1, 3, 90, **f), torch.zeros(1, 2, 16, 32, **f), 1)
    with pytest.raises(ValueError, match="contiguous"):
        binding.ida_rmsnorm(torch.zeros(4, 128, **f)[:, :64], torch.ones(64, **f))
    with pytest.raises(ValueError, match="group"):
        binding.ida_rmsnorm(torch.zeros(4, 96, **f), torch.ones(96, **f), group=64)
    with pytest.raises(binding.IdaError, match="groups"):
        binding.ida_rmsnorm(torch.zeros(4, 96, **f), torch.ones(96, **f), group=48)
    torch.cuda.synchronize()
    assert binding.ida_device_error() == 0
