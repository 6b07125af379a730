"""What the operators around the call refuse, on the CPU: the Python checks raise ValueError, the
library returns its status with nothing enqueued."""
import ctypes
import os
import subprocess

import pytest
import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import _binding as bind
from free_block_sparse_means_b200 import build as spr_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16
P = 4096  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    spr_build.build()
    return spr.load_library()


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype)


def test_struct_layouts_match_c(tmp_path):
    structs = {"spr_norm_rotate_params": spr.SprNormRotateParams,
               "spr_masked_params": spr.SprMaskedParams,
               "spr_project_params": spr.SprProjectParams}
    lines = []
    for c, py in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "probe.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"sparsepr.h\"\n"
                   "int main(void) {" + "\n".join(lines) + " return 0; }\n")
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    want = []
    for py in structs.values():
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want


# ------------------------------------------------------------ norm + rotation
def _nr(**kw):
    q = empty(2, 4, 10, 64)
    prm = spr.make_norm_rotate(q, q, q, q)
    for f, v in kw.items():
        setattr(prm, f, v)
    return prm


def _nr_call(lib, prm, Q=P, K=P, wq=None, wk=None, cos=P, sin=P, rows=10, pq=None, pk=None, Qo=P,
             Ko=P):
    return lib.sparsepr_norm_rotate(ctypes.byref(prm), Q, K, wq, wk, cos, sin, rows, pq, pk, Qo, Ko,
                                    None, None)


@pytest.mark.parametrize("fields,status", [
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Nq=0), 1), (dict(Nk=0), 1), (dict(Hk=-1), 1),
    (dict(d=0), 1), (dict(d=68), 2), (dict(d=264), 2), (dict(rot=-8), 1), (dict(rot=72), 1),
    (dict(rot=12), 2), (dict(rot=8, pairing=1), 2), (dict(pairing=2), 1), (dict(norm=2), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(dtype_in=3), 1), (dict(dtype_out=1), 2),
    (dict(dtype_in=1, dtype_out=2), 2), (dict(Nq=11), 1), (dict(B=40000), 2)])
def test_norm_rotate_parameters(lib, fields, status):
    assert _nr_call(lib, _nr(**fields)) == status


def test_norm_rotate_pointers_and_strides(lib):
    assert _nr_call(lib, _nr(), Q=None) == bind.SPR_EINVAL
    assert _nr_call(lib, _nr(), K=None) == bind.SPR_EINVAL
    assert _nr_call(lib, _nr(), Ko=None) == bind.SPR_EINVAL
    assert _nr_call(lib, _nr(), cos=None) == bind.SPR_EINVAL
    assert _nr_call(lib, _nr(), rows=0) == bind.SPR_EINVAL
    assert _nr_call(lib, _nr(norm=0), wq=P) == bind.SPR_EINVAL
    assert _nr_call(lib, _nr(), Q=P + 2) == bind.SPR_EUNSUPPORTED
    assert _nr_call(lib, _nr(), cos=P + 4) == bind.SPR_EUNSUPPORTED
    for field in ("q_strides", "k_strides", "qo_strides", "ko_strides"):
        prm = _nr()
        getattr(prm, field)[2] = 60
        assert _nr_call(lib, prm) == bind.SPR_EUNSUPPORTED, field
        prm = _nr()
        getattr(prm, field)[1] = -640
        assert _nr_call(lib, prm) == bind.SPR_EUNSUPPORTED, field
    prm = _nr()
    prm.qo_strides[0] = 0  # two batches written to one place
    assert _nr_call(lib, prm) == bind.SPR_EUNSUPPORTED


def test_norm_rotate_python_checks():
    q, k = empty(2, 4, 10, 64), empty(2, 2, 6, 64)
    prm = spr.make_norm_rotate(q, k, q, k)
    cos = empty(10, 32, dtype=torch.float32)
    ok = dict(cos=cos, sin=cos)
    for bad in (dict(cos=cos), dict(cos=cos, sin=cos[:, :31]), dict(cos=cos.double(), sin=cos),
                dict(ok, wq=empty(63)), dict(ok, wq=empty(64, dtype=torch.float32)),
                dict(ok, pos_q=empty(2, 9, dtype=torch.int32)),
                dict(ok, pos_k=empty(2, 6, dtype=torch.int64)),
                dict(ok, status=empty(3, dtype=torch.int32)), ok):  # the last: not on a GPU
        with pytest.raises(ValueError):
            spr.sparsepr_norm_rotate(prm, q, k, q, k, **bad)
    with pytest.raises(ValueError):  # another tensor than the parameters were made for
        spr.sparsepr_norm_rotate(prm, empty(2, 4, 11, 64), k, q, k, **ok)
    with pytest.raises(ValueError):
        spr.sparsepr_norm_rotate(prm, empty(2, 10, 4, 64).transpose(1, 2), k, q, k, **ok)
    with pytest.raises(ValueError):
        spr.sparsepr_norm_rotate(prm, q.half(), k, q, k, **ok)
    with pytest.raises(ValueError):
        spr.sparsepr_norm_rotate(spr.make_norm_rotate(q, None, q, None), q, k, q, k, **ok)
    for args, kw in (((q, None, q, q), {}), ((q, k, k, k), {}), ((q, k, q, q), {}),
                     ((q, empty(3, 2, 6, 64), q, empty(3, 2, 6, 64)), {}),
                     ((q, k.half(), q, k), {}), ((q[0], k, q[0], k), {}),
                     ((q.transpose(2, 3), k, q, k), {}), ((q.int(), None, q, None), {}),
                     ((q, k, q, k), dict(pairing="both"))):
        with pytest.raises(ValueError):
            spr.make_norm_rotate(*args, **kw)


# ----------------------------------------------------------- masked attention
def _am(**kw):
    q, k = empty(2, 4, 10, 64), empty(2, 2, 30, 64)
    prm = spr.make_masked(q, k, k, q)
    for f, v in kw.items():
        setattr(prm, f, v)
    return prm


def _am_call(lib, prm, Q=P, K=P, V=P, dq=None, dk=None, prefix=None, O=P, ws=P, n=1 << 40):
    return lib.sparsepr_attend_masked(ctypes.byref(prm), Q, K, V, None, dq, dk, prefix, None, O,
                                      None, ws, n, None, None)


@pytest.mark.parametrize("fields,status", [
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(Nq=0), 1),
    (dict(Nk=0), 1), (dict(d=96), 2), (dict(dtype=2), 1), (dict(scale=float("nan")), 1),
    (dict(softcap=-1.0), 1), (dict(softcap=float("inf")), 1), (dict(causal=2), 1),
    (dict(q_start=(1 << 30) + 1), 1), (dict(B=70000), 2)])
def test_masked_parameters(lib, fields, status):
    prm = _am(**fields)
    assert _am_call(lib, prm) == status
    assert lib.sparsepr_attend_masked_workspace(ctypes.byref(prm)) == 0
    with pytest.raises(spr.SparsePRError):
        spr.alloc_workspace(prm, device="cpu")


def test_masked_pointers_strides_and_workspace(lib):
    for kw in (dict(Q=None), dict(K=None), dict(V=None), dict(O=None), dict(dq=P), dict(dk=P),
               dict(prefix=P)):
        assert _am_call(lib, _am(), **kw) == bind.SPR_EINVAL, kw
    for kw in (dict(Q=P + 8), dict(V=P + 2), dict(O=P + 4)):
        assert _am_call(lib, _am(), **kw) == bind.SPR_EUNSUPPORTED, kw
    need = lib.sparsepr_attend_masked_workspace(ctypes.byref(_am()))
    assert need > 0
    for kw in (dict(ws=None), dict(ws=P + 16), dict(n=need - 1)):
        assert _am_call(lib, _am(), **kw) == bind.SPR_EWORKSPACE, kw
    for field in ("q_strides", "k_strides", "v_strides", "o_strides"):
        prm = _am()
        getattr(prm, field)[2] = 68
        assert _am_call(lib, prm) == bind.SPR_EUNSUPPORTED, field
    prm = _am()
    prm.o_strides[1] = 0
    assert _am_call(lib, prm) == bind.SPR_EUNSUPPORTED


def test_masked_python_checks():
    q, k = empty(2, 4, 10, 64), empty(2, 2, 30, 64)
    prm = spr.make_masked(q, k, k, q)
    ws = spr.alloc_workspace(prm, device="cpu")
    i32 = dict(dtype=torch.int32)
    for bad in (dict(k_len=empty(3, **i32)), dict(k_len=empty(2, dtype=torch.int64)),
                dict(doc_q=empty(2, 10, **i32)),
                dict(doc_q=empty(2, 10, **i32), doc_k=empty(2, 29, **i32)),
                dict(prefix=empty(2, **i32)), dict(slopes=empty(2, dtype=torch.float32)),
                dict(lse=empty(2, 4, 10)), dict()):  # the last: not on a GPU
        with pytest.raises(ValueError):
            spr.sparsepr_attend_masked(prm, q, k, k, q, ws, **bad)
    for args in ((q, k, k[:, :, :29], q), (q, k, k, q[:, :, :9]), (q, k.half(), k, q),
                 (q.float(), k.float(), k.float(), q.float()), (q, k[:1], k[:1], q),
                 (q.transpose(2, 3), k, k, q)):
        with pytest.raises(ValueError):
            spr.make_masked(*args)


# ----------------------------------------------------------------- projection
def _pj(**kw):
    prm = spr.make_project(empty(2, 3, 10, 64), empty(128, 192), empty(2, 2, 10, 64))
    for f, v in kw.items():
        setattr(prm, f, v)
    return prm


def _pj_call(lib, prm, X=P, W=P, R=None, Y=P, ws=P, n=1 << 40):
    return lib.sparsepr_project(ctypes.byref(prm), X, W, None, None, R, Y, ws, n, None, None)


@pytest.mark.parametrize("fields,status", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(Hx=0), 1), (dict(dy=0), 1), (dict(dx=100), 2),
    (dict(dx=72), 2), (dict(dy=72), 2), (dict(dtype=2), 1), (dict(act=4), 1), (dict(act=-1), 1),
    (dict(w_stride=196), 2), (dict(w_stride=184), 2), (dict(B=70000), 2), (dict(Hx=1 << 15), 2)])
def test_project_parameters(lib, fields, status):
    prm = _pj(**fields)
    assert _pj_call(lib, prm) == status
    assert lib.sparsepr_project_workspace(ctypes.byref(prm)) == 0
    with pytest.raises(spr.SparsePRError):
        spr.alloc_workspace(prm, device="cpu")


def test_project_pointers_strides_and_workspace(lib):
    for kw in (dict(X=None), dict(W=None), dict(Y=None)):
        assert _pj_call(lib, _pj(), **kw) == bind.SPR_EINVAL, kw
    for kw in (dict(X=P + 8), dict(W=P + 2), dict(Y=P + 4), dict(R=P + 4)):
        assert _pj_call(lib, _pj(), **kw) == bind.SPR_EUNSUPPORTED, kw
    need = lib.sparsepr_project_workspace(ctypes.byref(_pj()))
    assert need > 0
    for kw in (dict(ws=None), dict(ws=P + 16), dict(n=need - 1)):
        assert _pj_call(lib, _pj(), **kw) == bind.SPR_EWORKSPACE, kw
    for field in ("x_strides", "y_strides"):
        prm = _pj()
        getattr(prm, field)[2] = 68
        assert _pj_call(lib, prm) == bind.SPR_EUNSUPPORTED, field
    prm = _pj()
    prm.y_strides[1] = 0
    assert _pj_call(lib, prm) == bind.SPR_EUNSUPPORTED


def test_project_python_checks():
    x, w, y = empty(2, 3, 10, 64), empty(128, 192), empty(2, 2, 10, 64)
    prm = spr.make_project(x, w, y)
    ws = spr.alloc_workspace(prm, device="cpu")
    for bad in (dict(bias=empty(127)), dict(bias=empty(128, dtype=torch.float32)),
                dict(gate=empty(128)), dict(residual=y[:, :, :9]),
                dict(residual=empty(2, 10, 2, 64).transpose(1, 2)), dict()):
        with pytest.raises(ValueError):
            spr.sparsepr_project(prm, x, w, y, ws, **bad)
    with pytest.raises(ValueError):
        spr.sparsepr_project(prm, x, w[:, :64], y, ws)
    for args, kw in (((x, w[:127], y), {}), ((x, w.half(), y), {}), ((x, w.t().contiguous().t(), y), {}),
                     ((x, w, y[:, :, :9]), {}), ((x, w, y), dict(act="relu")),
                     ((x, w, y), dict(residual=y[:1]))):
        with pytest.raises(ValueError):
            spr.make_project(*args, **kw)


def test_gradients_are_refused():
    """Forward only: an input that requires a gradient is not silently cut off."""
    x, w, y = empty(2, 3, 10, 64), empty(128, 192).requires_grad_(), empty(2, 2, 10, 64)
    prm = spr.make_project(x, w, y)
    ws = spr.alloc_workspace(prm, device="cpu")
    with pytest.raises(ValueError, match="no backward"):
        spr.sparsepr_project(prm, x, w, y, ws)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        spr.sparsepr_project(prm, x, w, y, ws)
