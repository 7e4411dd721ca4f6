"""Host side of the RMS norm and the linear attention, without a GPU: struct layouts, refusals before
anything is queued (fake addresses, never dereferenced), workspace sizes, the bindings' own checks."""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

from pooled_selective_scan_b200 import _call, linattn, rmsnorm  # noqa: E402
from pooled_selective_scan_b200 import _native as nat  # noqa: E402
from pooled_selective_scan_b200 import build as fvbuild  # noqa: E402

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fastvim_ssm.h")
FAKE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    fvbuild.build()
    return nat.lib()


def fill(a, names):
    for i, n in enumerate(names):
        setattr(a, n, FAKE + (i << 34))
    return a


def change(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def norm_args(**kw):
    a = fill(nat.FvRmsnormArgs(), ("x", "weight", "y"))
    a.M, a.E, a.eps, a.x_type, a.y_type = 100, 768, 1e-5, nat.FV_TYPE_BF16, nat.FV_TYPE_BF16
    return change(a, kw)


def norm_grad_args(**kw):
    a = fill(nat.FvRmsnormGradArgs(), ("s", "dy", "weight", "dx", "dweight"))
    a.M, a.E, a.eps, a.s_type, a.y_type = 100, 768, 1e-5, nat.FV_TYPE_F32, nat.FV_TYPE_BF16
    return change(a, kw)


def attn_args(**kw):
    a = fill(nat.FvLinattnArgs(), ("q", "k", "v", "g", "y"))
    a.N, a.T, a.H, a.Hk, a.dk, a.dv, a.type, a.scale = 2, 300, 4, 2, 64, 64, nat.FV_TYPE_BF16, 0.125
    return change(a, kw)


def attn_grads(**kw):
    g = nat.FvLinattnGrads()
    for i, n in enumerate(("dy", "dq", "dk", "dv", "dg")):
        setattr(g, n, FAKE + ((20 + i) << 34))
    return change(g, kw)


def step_args(**kw):
    a = fill(nat.FvLinattnStepArgs(), ("q", "k", "v", "g", "state", "y"))
    a.B, a.S, a.H, a.Hk, a.dk, a.dv, a.type, a.scale = 3, 3, 4, 2, 64, 64, nat.FV_TYPE_F32, 0.125
    return change(a, kw)


def test_structs_and_constants_match_the_header(tmp_path):
    structs = {"fv_rmsnorm_args": nat.FvRmsnormArgs, "fv_rmsnorm_grad_args": nat.FvRmsnormGradArgs,
               "fv_linattn_args": nat.FvLinattnArgs, "fv_linattn_grads": nat.FvLinattnGrads,
               "fv_linattn_step_args": nat.FvLinattnStepArgs}
    consts = ["FV_TYPE_F32", "FV_TYPE_BF16", "FV_TYPE_F16", "FV_TYPE_E4M3", "FV_LA_HEAD_DECAY"]
    lines, want = [], []
    for c in consts:
        lines.append(f'printf("%d\\n", (int){c});')
        want.append(getattr(nat, c))
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    src = tmp_path / "abi.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fastvim_ssm.h"\nint main(void){' + "\n".join(lines) + "return 0;}\n")
    exe = tmp_path / "abi"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    assert [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()] == want


R = FAKE + (9 << 34)
NORM_BAD = [
    (dict(M=-1), nat.FV_ERR_SHAPE), (dict(E=0), nat.FV_ERR_SHAPE), (dict(E=766), nat.FV_ERR_SHAPE),
    (dict(E=16388), nat.FV_ERR_UNSUPPORTED), (dict(M=1 << 31), nat.FV_ERR_UNSUPPORTED),
    (dict(eps=0.0), nat.FV_ERR_SHAPE), (dict(eps=float("nan")), nat.FV_ERR_SHAPE), (dict(eps=float("inf")), nat.FV_ERR_SHAPE),
    (dict(x_type=nat.FV_TYPE_E4M3), nat.FV_ERR_SHAPE), (dict(y_type=nat.FV_TYPE_F32), nat.FV_ERR_SHAPE),
    (dict(x=None), nat.FV_ERR_NULL), (dict(weight=None), nat.FV_ERR_NULL), (dict(y=None), nat.FV_ERR_NULL),
    (dict(x=FAKE + 8), nat.FV_ERR_ALIGN), (dict(x_stride=700), nat.FV_ERR_SHAPE), (dict(x_stride=770), nat.FV_ERR_SHAPE),
    (dict(residual=R, res_type=nat.FV_TYPE_F16, s=R + (1 << 33)), nat.FV_ERR_SHAPE), (dict(residual=R, res_type=nat.FV_TYPE_F32), nat.FV_ERR_NULL),
    (dict(s=R), nat.FV_ERR_SHAPE), (dict(scales=R), nat.FV_ERR_SHAPE), (dict(y_type=nat.FV_TYPE_E4M3), nat.FV_ERR_NULL),
    (dict(block=128), nat.FV_ERR_SHAPE), (dict(block=64, y_type=nat.FV_TYPE_E4M3, scales=R), nat.FV_ERR_SHAPE),
    (dict(E=132, block=128, y_type=nat.FV_TYPE_E4M3, scales=R), nat.FV_ERR_SHAPE),
    (dict(y=FAKE), nat.FV_ERR_ALIAS), (dict(residual=R, res_type=nat.FV_TYPE_F32, s=R + 16), nat.FV_ERR_ALIAS),
    (dict(residual=R, res_type=nat.FV_TYPE_F32, s=FAKE + (2 << 34)), nat.FV_ERR_ALIAS),
]


@pytest.mark.parametrize("kw,status", NORM_BAD)
def test_norm_refusals(lib, kw, status):
    assert lib.fastvim_rmsnorm_validate(ctypes.byref(norm_args(**kw))) == status
    assert lib.fastvim_rmsnorm_forward(ctypes.byref(norm_args(**kw)), None) == status


def test_norm_accepts(lib):
    for kw in (dict(), dict(residual=R, res_type=nat.FV_TYPE_F32, s=R), dict(y_type=nat.FV_TYPE_E4M3, scales=R),
               dict(y_type=nat.FV_TYPE_E4M3, scales=R, block=128), dict(x_stride=1600), dict(M=0, x=None, y=None)):
        assert lib.fastvim_rmsnorm_validate(ctypes.byref(norm_args(**kw))) == nat.FV_OK
    assert lib.fastvim_rmsnorm_validate(None) == nat.FV_ERR_NULL
    assert lib.fastvim_rmsnorm_forward(ctypes.byref(norm_args(M=0, x=None, y=None)), None) == nat.FV_OK


@pytest.mark.parametrize("kw,status", [
    (dict(E=6), nat.FV_ERR_SHAPE), (dict(y_type=nat.FV_TYPE_E4M3), nat.FV_ERR_SHAPE), (dict(s_type=nat.FV_TYPE_F16), nat.FV_ERR_SHAPE),
    (dict(eps=-1.0), nat.FV_ERR_SHAPE), (dict(dy=None), nat.FV_ERR_NULL), (dict(dweight=None), nat.FV_ERR_NULL),
    (dict(dx=FAKE), nat.FV_ERR_ALIAS), (dict(dresidual=FAKE + (3 << 34)), nat.FV_ERR_ALIAS), (dict(s=FAKE + 4), nat.FV_ERR_ALIGN)])
def test_norm_gradient_refusals(lib, kw, status):
    ws = ctypes.c_void_p(FAKE + (30 << 34))
    assert lib.fastvim_rmsnorm_backward(ctypes.byref(norm_grad_args(**kw)), ws, 1 << 30, None) == status


def test_norm_gradient_workspace(lib):
    a = norm_grad_args()
    need = lib.fastvim_rmsnorm_backward_workspace_size(ctypes.byref(a))
    assert need >= 100 * 768 * 4 // 8 and need % 256 == 0
    assert lib.fastvim_rmsnorm_backward(ctypes.byref(a), None, need, None) == nat.FV_ERR_WORKSPACE
    assert lib.fastvim_rmsnorm_backward(ctypes.byref(a), ctypes.c_void_p(FAKE + (30 << 34)), need - 1, None) == nat.FV_ERR_WORKSPACE
    assert lib.fastvim_rmsnorm_backward(ctypes.byref(a), ctypes.c_void_p(FAKE + (30 << 34) + 16), need, None) == nat.FV_ERR_WORKSPACE
    assert lib.fastvim_rmsnorm_backward_workspace_size(ctypes.byref(norm_grad_args(E=6))) == 0


ATTN_BAD = [
    (dict(N=-1), nat.FV_ERR_SHAPE), (dict(T=-1), nat.FV_ERR_SHAPE), (dict(Hk=3), nat.FV_ERR_SHAPE), (dict(Hk=0), nat.FV_ERR_SHAPE),
    (dict(dk=12), nat.FV_ERR_SHAPE), (dict(dv=0), nat.FV_ERR_SHAPE), (dict(dk=136), nat.FV_ERR_UNSUPPORTED),
    (dict(dv=264), nat.FV_ERR_UNSUPPORTED), (dict(type=nat.FV_TYPE_F16), nat.FV_ERR_SHAPE), (dict(flags=2), nat.FV_ERR_SHAPE),
    (dict(scale=float("nan")), nat.FV_ERR_SHAPE), (dict(q_stride=64), nat.FV_ERR_SHAPE), (dict(k_stride=132), nat.FV_ERR_SHAPE),
    (dict(g_stride=3), nat.FV_ERR_SHAPE), (dict(g_stride=8, flags=1), nat.FV_ERR_SHAPE), (dict(N=1 << 20, T=1 << 12), nat.FV_ERR_UNSUPPORTED),
    (dict(q=None), nat.FV_ERR_NULL), (dict(g=None), nat.FV_ERR_NULL), (dict(v=FAKE + 8), nat.FV_ERR_ALIGN),
    (dict(g=FAKE + (3 << 34) + 2), nat.FV_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", ATTN_BAD + [
    (dict(y=None), nat.FV_ERR_NULL), (dict(y=FAKE + 1024), nat.FV_ERR_ALIAS), (dict(final_state=FAKE + (4 << 34)), nat.FV_ERR_ALIAS),
    (dict(initial_state=R, final_state=R + 16), nat.FV_ERR_ALIAS)])
def test_attention_refusals(lib, kw, status):
    a = attn_args(**kw)
    assert lib.fastvim_linattn_validate(ctypes.byref(a)) == status
    assert lib.fastvim_linattn_forward(ctypes.byref(a), ctypes.c_void_p(FAKE + (40 << 34)), 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", ATTN_BAD)
def test_attention_gradient_refusals(lib, kw, status):
    assert lib.fastvim_linattn_backward(ctypes.byref(attn_args(**kw)), ctypes.byref(attn_grads()),
                                        ctypes.c_void_p(FAKE + (40 << 34)), 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), nat.FV_ERR_NULL), (dict(dq=None), nat.FV_ERR_NULL), (dict(dg=None), nat.FV_ERR_NULL),
    (dict(dv=FAKE + 8), nat.FV_ERR_ALIGN), (dict(dq=FAKE), nat.FV_ERR_ALIAS), (dict(dk=FAKE + (21 << 34)), nat.FV_ERR_ALIAS)])
def test_attention_gradient_outputs(lib, kw, status):
    assert lib.fastvim_linattn_backward(ctypes.byref(attn_args()), ctypes.byref(attn_grads(**kw)),
                                        ctypes.c_void_p(FAKE + (40 << 34)), 1 << 40, None) == status


def test_attention_workspaces(lib):
    """A dense call that fills the card needs a status word only; few heads over a long sequence are cut
    into pieces with a state each; the gradient keeps two states a chunk."""
    size = lambda **kw: lib.fastvim_linattn_workspace_size(ctypes.byref(attn_args(**kw)))  # noqa: E731
    grad = lambda **kw: lib.fastvim_linattn_backward_workspace_size(ctypes.byref(attn_args(**kw)))  # noqa: E731
    assert size(N=64, H=12, Hk=12) == 256
    assert size(N=1, T=65536, H=2) > 256 + 2 * 64 * 64 * 4 * 4
    assert size(cu_seqlens=FAKE + (8 << 34), N=40, T=5000) > 256
    assert grad(N=1, T=1024, H=4) > 2 * 8 * 4 * 64 * 64 * 4
    assert grad(N=1, T=1024, H=4) < grad(N=1, T=2048, H=4)
    assert size(dk=12) == 0 and grad(dk=12) == 0
    a = attn_args()
    for ws, n in ((None, 1 << 40), (FAKE + (40 << 34), 255), (FAKE + (40 << 34) + 128, 1 << 40)):
        assert lib.fastvim_linattn_forward(ctypes.byref(a), ctypes.c_void_p(ws), n, None) == nat.FV_ERR_WORKSPACE
        assert lib.fastvim_linattn_backward(ctypes.byref(a), ctypes.byref(attn_grads()), ctypes.c_void_p(ws), n, None) == nat.FV_ERR_WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), nat.FV_ERR_SHAPE), (dict(S=2), nat.FV_ERR_SHAPE), (dict(dk=136), nat.FV_ERR_UNSUPPORTED), (dict(state=None), nat.FV_ERR_NULL),
    (dict(q=None), nat.FV_ERR_NULL), (dict(q_stride=130), nat.FV_ERR_SHAPE), (dict(v=FAKE + 4), nat.FV_ERR_ALIGN),
    (dict(slots=R + 2), nat.FV_ERR_ALIGN), (dict(y=FAKE + (4 << 34)), nat.FV_ERR_ALIAS), (dict(state=FAKE), nat.FV_ERR_ALIAS),
    (dict(status=FAKE + (5 << 34)), nat.FV_ERR_ALIAS)])
def test_step_refusals(lib, kw, status):
    assert lib.fastvim_linattn_step(ctypes.byref(step_args(**kw)), None) == status


def test_null_structs(lib):
    assert lib.fastvim_linattn_validate(None) == nat.FV_ERR_NULL
    assert lib.fastvim_linattn_workspace_size(None) == 0
    assert lib.fastvim_linattn_step(None, None) == nat.FV_ERR_NULL
    assert lib.fastvim_rmsnorm_backward(None, None, 0, None) == nat.FV_ERR_NULL
    assert lib.fastvim_linattn_backward(ctypes.byref(attn_args()), None, ctypes.c_void_p(FAKE), 0, None) == nat.FV_ERR_NULL


# ---- the bindings' checks -----------------------------------------------------------------------------


def test_host_tensors_and_types_are_refused():
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        rmsnorm.forward(x, w)
    with pytest.raises(TypeError):
        rmsnorm.forward(x.double(), w)
    with pytest.raises(TypeError):
        rmsnorm.forward(None, w)
    with pytest.raises(ValueError, match="CUDA"):
        rmsnorm.backward(x, w, x)
    q = torch.zeros(1, 3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        linattn.forward(q, q, q, torch.zeros(1, 3, 2))
    with pytest.raises(TypeError):
        linattn.forward(q.half(), q.half(), q.half(), torch.zeros(1, 3, 2))
    with pytest.raises(ValueError, match="CUDA"):
        linattn.step(q[0], q[0], q[0], torch.zeros(3, 2), torch.zeros(3, 2, 64, 64))


def test_token_strides():
    wide = torch.zeros(2, 5, 40)
    assert _call.token_stride("t", wide[..., :16].unflatten(-1, (2, 8)), 2) == 40
    assert _call.token_stride("t", wide, 2, 1) == 0
    assert _call.token_stride("t", wide[:, :1, :16].unflatten(-1, (2, 8)), 2) == 200
    assert _call.token_stride("t", wide[:1, :1, :16].unflatten(-1, (2, 8)), 2) == 0
    with pytest.raises(ValueError, match="constant step"):
        _call.token_stride("t", wide[:, :4, :16].unflatten(-1, (2, 8)), 2)
    with pytest.raises(ValueError, match="overlap"):
        _call.token_stride("t", torch.zeros(1, 1, 2, 8).expand(2, 5, 2, 8), 2)
    with pytest.raises(ValueError, match="one token"):
        _call.token_stride("t", torch.zeros(2, 5, 8, 2).transpose(-1, -2), 2)


def test_sizes_that_32_bits_do_not_hold_are_refused():
    assert _call.count("rows", 2**31 - 1) == 2**31 - 1
    for n in (2**31, 2**32, 2**32 + 1536):
        with pytest.raises(ValueError, match="rows must be below 2"):
            _call.count("rows", n)
    with pytest.raises(ValueError, match="channels"):
        rmsnorm.backward_workspace_size(5, 2**32 + 1536)
