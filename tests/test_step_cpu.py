"""Host-side checks of the operators around the expert products (no GPU): the C
ABI's refusals, the sizes of plans, the Python layer's refusals on stand-ins for
CUDA tensors, and the 64-bit implementations that the GPU tests compare with."""
import ctypes
from array import array

import numpy as np
import pytest
import torch

import moe_ragged_contraction_gb300 as mx
from moe_ragged_contraction_gb300 import _lib, experts
import _step_ref as R

P = 0x10000  # 256-byte aligned fake address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    mx.build()
    return mx.load()


def plan(lib, ids=P, id_type=0, T=8, k=2, first=0, local=4, align=32, rows=128, offs=P, slot=P, src=P):
    return lib.mxfp8_token_plan(ids, id_type, T, k, first, local, align, rows, offs, slot, src, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), _lib.EINVAL), (dict(k=0), _lib.EINVAL), (dict(k=65), _lib.EINVAL), (dict(T=2 ** 30), _lib.EINVAL), (dict(T=2 ** 62), _lib.EINVAL),
    (dict(id_type=2), _lib.EINVAL), (dict(first=-1), _lib.EINVAL), (dict(local=0), _lib.EINVAL), (dict(local=2049), _lib.EINVAL),
    (dict(align=0), _lib.EINVAL), (dict(align=1025), _lib.EINVAL), (dict(rows=-32), _lib.EINVAL), (dict(rows=100), _lib.EINVAL),
    (dict(rows=2 ** 31), _lib.EINVAL), (dict(ids=None), _lib.EINVAL), (dict(offs=None), _lib.EINVAL), (dict(slot=None), _lib.EINVAL),
    (dict(src=None), _lib.EINVAL), (dict(ids=P + 2), _lib.EALIGN), (dict(id_type=1, ids=P + 4), _lib.EALIGN), (dict(offs=P + 1), _lib.EALIGN),
    (dict(slot=P + 2), _lib.EALIGN), (dict(src=P + 3), _lib.EALIGN),
])
def test_plan_validation(lib, kw, code):
    assert plan(lib, **kw) == code and len(lib.mxfp8_last_error()) > 0


def rows_call(lib, name, T=8, H=64, k=2, rows=128, tok=P, srt=P, slot=P, src=P, extra=P):
    calls = {
        "dispatch": lambda: lib.mxfp8_token_dispatch(tok, T, H, k, slot, src, rows, srt, None),
        "dispatch_mxfp8": lambda: lib.mxfp8_token_dispatch_mxfp8(tok, T, H, k, slot, src, rows, srt, extra, None),
        "dispatch_grad": lambda: lib.mxfp8_token_dispatch_grad(srt, rows, T, H, k, slot, tok, None),
        "combine": lambda: lib.mxfp8_token_combine(srt, rows, extra, T, H, k, slot, tok, None),
        "combine_grad": lambda: lib.mxfp8_token_combine_grad(tok, srt, extra, T, H, k, slot, src, rows, srt, extra, None),
    }
    return calls[name]()


ROW_OPS = ["dispatch", "dispatch_mxfp8", "dispatch_grad", "combine", "combine_grad"]


@pytest.mark.parametrize("name", ROW_OPS)
@pytest.mark.parametrize("kw", [dict(T=-1), dict(k=0), dict(k=65), dict(T=2 ** 30), dict(H=0), dict(H=32800), dict(H=-8), dict(H=44), dict(rows=-1),
                                dict(rows=2 ** 31), dict(tok=None), dict(srt=None), dict(slot=None), dict(tok=P + 8), dict(srt=P + 2), dict(slot=P + 2)])
def test_row_operator_validation(lib, name, kw):
    assert rows_call(lib, name, **kw) in (_lib.EINVAL, _lib.EALIGN) and len(lib.mxfp8_last_error()) > 0


def test_row_operator_validation_of_single_arguments(lib):
    assert rows_call(lib, "dispatch_mxfp8", H=40) == _lib.EINVAL
    for name in ("dispatch", "dispatch_mxfp8", "combine_grad"):
        assert rows_call(lib, name, src=None) == _lib.EINVAL and rows_call(lib, name, src=P + 1) == _lib.EALIGN
    for name in ("dispatch_mxfp8", "combine", "combine_grad"):
        assert rows_call(lib, name, extra=None) == _lib.EINVAL
    for name in ("combine", "combine_grad"):
        assert rows_call(lib, name, extra=P + 2) == _lib.EALIGN


@pytest.mark.parametrize("T,k,local,align", [(1, 1, 1, 32), (1, 2, 4, 32), (5, 3, 2, 7), (100, 4, 9, 1), (0, 2, 4, 32), (3, 2, 100, 128)])
def test_plan_rows_hold_the_worst_routing_and_no_more(T, k, local, align):
    mx.build()
    rows = mx.token_plan_rows(T, k, local, align)
    assert rows % align == 0
    # the worst routing: one pair for as many experts as there are, the rest to one of them
    ids = np.full(T * k, 0)
    used = min(local, T * k)
    ids[:used] = np.arange(used)
    need = 0
    for extra in range(align):  # the last expert's count can be anything
        counts = np.bincount(ids, minlength=local)
        moved = min(extra, counts[0] - 1) if used > 1 else 0
        if T * k:
            counts[0] -= moved
            counts[used - 1] += moved
        need = max(need, int(((counts + align - 1) // align * align).sum()))
    assert need <= rows <= need + align
    with pytest.raises(ValueError):
        mx.token_plan_rows(-1, k, local, align)
    with pytest.raises(ValueError):
        mx.token_plan_rows(2 ** 32 + T, k, local, align)
    with pytest.raises(ValueError):
        mx.token_plan_rows(T, k, local + 2 ** 32, align)


def grads_call(lib, name="clip", ptrs=(P, P + 4096), sizes=(8, 8), types=(0, 1), n=None, norm=P, norm_in=None, outs=None, max_norm=1.0, eps=1e-6, ws=()):
    a, b, c = array("Q", [p or 0 for p in ptrs]), array("q", sizes), array("i", types)
    o = array("Q", [p or 0 for p in outs]) if outs is not None else None
    at = lambda v: v.buffer_info()[0] if v is not None and len(v) else None  # noqa: E731
    n = len(ptrs) if n is None else n
    if name == "norm":
        f = lib.mxfp8_grad_norm_ws if ws else lib.mxfp8_grad_norm
        return f(at(a), at(b), at(c), n, norm, *ws, None)
    f = lib.mxfp8_clip_grads_ws if ws else lib.mxfp8_clip_grads
    return f(at(a), at(b), at(c), n, max_norm, eps, norm_in, norm, at(o), *ws, None)


@pytest.mark.parametrize("name", ["norm", "clip"])
@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), _lib.EINVAL), (dict(n=65537), _lib.EINVAL), (dict(types=(0, 2)), _lib.EINVAL), (dict(sizes=(8, -1)), _lib.EINVAL),
    (dict(sizes=(8, 2 ** 50)), _lib.EINVAL), (dict(ptrs=(P, None)), _lib.EINVAL), (dict(ptrs=(P + 1, P + 4096)), _lib.EALIGN),
    (dict(ptrs=(P, P + 4098)), _lib.EALIGN), (dict(norm=P + 2), _lib.EALIGN), (dict(ws=(None, 1 << 20)), _lib.EINVAL),
    (dict(ws=(P + 16, 1 << 20)), _lib.EALIGN), (dict(ws=(P, 8)), _lib.ENOWS),
])
def test_gradient_list_validation(lib, name, kw, code):
    assert grads_call(lib, name, **kw) == code and len(lib.mxfp8_last_error()) > 0


@pytest.mark.parametrize("kw,code", [
    (dict(max_norm=-1.0), _lib.EINVAL), (dict(max_norm=float("inf")), _lib.EINVAL), (dict(max_norm=float("nan")), _lib.EINVAL),
    (dict(eps=-1.0), _lib.EINVAL), (dict(eps=float("nan")), _lib.EINVAL), (dict(norm_in=P + 64), _lib.EINVAL), (dict(norm_in=P + 2, norm=None), _lib.EALIGN),
    (dict(outs=(P, None)), _lib.EINVAL), (dict(outs=(P, P + 4097)), _lib.EALIGN),
    # overlaps: the same tensor twice, views that share elements, an output over another gradient or output or shifted over its own
    (dict(ptrs=(P, P)), _lib.EINVAL), (dict(ptrs=(P, P + 12)), _lib.EINVAL), (dict(ptrs=(P + 16, P)), _lib.EINVAL),
    (dict(outs=(P + 4096, P + 8192)), _lib.EINVAL), (dict(outs=(P + 8192, P + 8200)), _lib.EINVAL), (dict(outs=(P + 2, P + 8192)), _lib.EINVAL),
    (dict(ptrs=(P, P), outs=(P + 8192, P)), _lib.EINVAL),
])
def test_clip_validation(lib, kw, code):
    assert grads_call(lib, "clip", **kw) == code


def test_lists_that_are_fine_get_past_the_checks(lib):
    """No device here: what passes the checks ends at the device's."""
    if torch.cuda.is_available():
        pytest.skip("a device would run these")
    past = (_lib.ECUDA, _lib.EUNSUPPORTED)
    for kw in (dict(), dict(ptrs=(P, P + 16)), dict(outs=(P + 8192, P + 4096)), dict(ptrs=(P, P), outs=(P + 8192, P + 16384)), dict(ptrs=(P, None), sizes=(8, 0)),
               dict(ptrs=(P + 4096, P), outs=(P + 4096, P)), dict(norm_in=P), dict(norm=None)):
        assert grads_call(lib, "clip", **kw) in past, kw
    assert grads_call(lib, "norm", ptrs=(P, P)) in past and grads_call(lib, "norm", ptrs=(), sizes=(), types=()) in past
    assert plan(lib) in past and plan(lib, T=0, ids=None, slot=None) in past and plan(lib, rows=0, src=None) in past
    for name in ROW_OPS:
        assert rows_call(lib, name) in past, name


def test_grad_workspace(lib):
    f = lib.mxfp8_grad_workspace_bytes
    assert f(-1) == 0 and f(65537) == 0 and f(0) > 0 and f(5000) > f(1)
    assert mx.grad_workspace_bytes(2 ** 32 + 1) == 0 and mx.grad_workspace_bytes(3) == f(3)


# ------------------------------------------------------------------ the Python layer, on stand-ins

class Host(torch.Tensor):
    """A host tensor that passes for one on cuda:0 (or on `dev`)."""
    dev = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.dev


def t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype).as_subclass(Host)


def elsewhere(v):
    class Other(Host):
        dev = 1
    return v.as_subclass(Other)


@pytest.fixture
def asked(monkeypatch):
    """The names of the library's functions that were called; none computes anything."""
    names = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: names.append(name) or 0

    monkeypatch.setattr(_lib, "_lib", Library())
    monkeypatch.setattr(experts, "_torch", torch)
    monkeypatch.setattr(experts, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return names


bf, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
T, K, H, E, ROWS = 6, 2, 64, 3, 96


def token_plan():
    return mx.TokenPlan(t(i32, E), t(i32, T, K), t(i32, ROWS))


def op(name, **kw):
    p = kw.pop("plan", None) or token_plan()
    args = {
        "token_plan": dict(ids=t(i32, T, K), local=E, rows=ROWS, out=token_plan()),
        "token_dispatch": dict(x=t(bf, T, H), plan=p, out=t(bf, ROWS, H)),
        "token_dispatch_mxfp8": dict(x=t(bf, T, H), plan=p, q=t(u8, ROWS, H), s=t(u8, ROWS, H // 32)),
        "token_dispatch_grad": dict(dxs=t(bf, ROWS, H), plan=p, out=t(bf, T, H)),
        "token_combine": dict(y=t(bf, ROWS, H), weights=t(f32, T, K), plan=p, out=t(bf, T, H)),
        "token_combine_grad": dict(dout=t(bf, T, H), y=t(bf, ROWS, H), weights=t(f32, T, K), plan=p, dy=t(bf, ROWS, H), dweights=t(f32, T, K)),
        "grad_norm": dict(grads=[t(bf, 4, 5), t(f32, 7)], out=t(f32)),
        "clip_grads": dict(grads=[t(bf, 4, 5), t(f32, 7)], max_norm=1.0, norm=t(f32), out=[t(bf, 4, 5), t(f32, 7)]),
    }[name]
    return getattr(mx, name)(**{**args, **kw})


OPS = ["token_plan", "token_dispatch", "token_dispatch_mxfp8", "token_dispatch_grad", "token_combine", "token_combine_grad", "grad_norm", "clip_grads"]


@pytest.mark.parametrize("name", OPS)
def test_calls_reach_the_library(asked, name):
    op(name)
    assert asked == ["mxfp8_" + name]


@pytest.mark.parametrize("name,kw", [
    ("token_plan", dict(ids=t(f32, T, K))), ("token_plan", dict(ids=t(i32, T))), ("token_plan", dict(local=2 ** 32 + E)), ("token_plan", dict(rows=2 ** 32)),
    ("token_plan", dict(first_expert=2 ** 32)), ("token_plan", dict(align=2 ** 32 + 32)), ("token_plan", dict(rows=64)), ("token_plan", dict(rows=-32, out=None)),
    ("token_plan", dict(ids=t(i32, K, T).T)),
    ("token_dispatch", dict(x=t(f32, T, H))), ("token_dispatch", dict(x=t(bf, T + 1, H))), ("token_dispatch", dict(x=t(bf, H, T).T)), ("token_dispatch", dict(out=t(bf, ROWS, H + 8))),
    ("token_dispatch", dict(x=t(bf))), ("token_dispatch", dict(x=elsewhere(t(bf, T, H)))), ("token_dispatch", dict(out=elsewhere(t(bf, ROWS, H)))),
    ("token_dispatch_mxfp8", dict(q=t(bf, ROWS, H))), ("token_dispatch_mxfp8", dict(s=t(u8, ROWS, H))),
    ("token_dispatch_grad", dict(dxs=t(bf, ROWS + 1, H))), ("token_dispatch_grad", dict(out=t(f32, T, H))),
    ("token_combine", dict(weights=t(bf, T, K))), ("token_combine", dict(weights=t(f32, T, K + 1))), ("token_combine", dict(y=t(bf, ROWS - 1, H))),
    ("token_combine", dict(weights=elsewhere(t(f32, T, K)))),
    ("token_combine_grad", dict(y=t(bf, ROWS, H + 8))), ("token_combine_grad", dict(dy=t(bf, T, H))), ("token_combine_grad", dict(dweights=t(f32, K, T))),
    ("grad_norm", dict(grads=[], out=None)), ("clip_grads", dict(grads=[], out=None, norm=None)), ("grad_norm", dict(grads=t(bf, 4, 5))), ("grad_norm", dict(grads=[t(torch.float16, 4)])), ("grad_norm", dict(grads=[t(bf, 4, 6).T])),
    ("grad_norm", dict(grads=[t(bf, 4), elsewhere(t(bf, 4))])), ("grad_norm", dict(out=t(f32, 1))), ("grad_norm", dict(out=t(bf))), ("grad_norm", dict(grads=[t(bf, 4), None])),
    ("clip_grads", dict(out=[t(bf, 4, 5)])), ("clip_grads", dict(out=[t(bf, 5, 4), t(f32, 7)])), ("clip_grads", dict(out=[t(f32, 4, 5), t(f32, 7)])),
    ("clip_grads", dict(norm=t(f32, 2))), ("clip_grads", dict(norm=elsewhere(t(f32)))), ("clip_grads", dict(workspace=t(f32, 4096))),
])
def test_refusals(asked, name, kw):
    with pytest.raises((ValueError, TypeError)):
        op(name, **kw)
    assert not asked


@pytest.mark.parametrize("name", OPS[1:6])
@pytest.mark.parametrize("bad", [mx.TokenPlan(t(i32, E), t(i32, T), t(i32, ROWS)), mx.TokenPlan(t(i32, E), t(i64, T, K), t(i32, ROWS)), mx.TokenPlan(t(i32, E), t(i32, T, K), t(f32, ROWS)),
                                 mx.TokenPlan(t(i32, E), t(i32, T, K), elsewhere(t(i32, ROWS))), mx.TokenPlan(None, None, None), mx.TokenPlan(t(i32, E), t(i32, T, K), t(i32, 2 * ROWS)[::2])])
def test_plans_that_are_none(asked, name, bad):
    with pytest.raises((ValueError, TypeError)):
        op(name, plan=bad)
    assert not asked


@pytest.mark.parametrize("name,key,make", [
    ("token_dispatch", "x", lambda: t(bf, T, H)), ("token_dispatch_mxfp8", "x", lambda: t(bf, T, H)), ("token_dispatch_grad", "dxs", lambda: t(bf, ROWS, H)),
    ("token_combine", "y", lambda: t(bf, ROWS, H)), ("token_combine", "weights", lambda: t(f32, T, K)), ("token_combine", "out", lambda: t(bf, T, H)),
    ("token_combine_grad", "dout", lambda: t(bf, T, H)), ("token_combine_grad", "weights", lambda: t(f32, T, K)), ("token_combine_grad", "dy", lambda: t(bf, ROWS, H)),
])
def test_tensors_that_require_a_gradient(asked, name, key, make):
    v = make().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        op(name, **{key: v})
    assert not asked
    with torch.no_grad():
        op(name, **{key: v})
    op(name, **{key: v.detach()})
    assert len(asked) == 2


@pytest.mark.parametrize("name", ["grad_norm", "clip_grads"])
def test_lists_with_a_tensor_that_requires_a_gradient(asked, name):
    v = t(bf, 4, 5).requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        op(name, grads=[v, t(f32, 7)])
    assert not asked
    with torch.no_grad():
        op(name, grads=[v, t(f32, 7)])
    assert len(asked) == 1


# ------------------------------------------------------------------ the 64-bit implementations

def test_reference_plan_by_hand():
    ids = np.array([[2, 0], [2, 5], [-1, 2], [0, 0]])
    offs, slot, src, dropped = R.plan(ids, 0, 3, 2, 8)
    assert offs.tolist() == [4, 4, 8] and dropped == 0
    assert slot.tolist() == [[4, 0], [5, -1], [-1, 6], [1, 2]]
    assert src.tolist() == [1, 6, 7, -1, 0, 2, 5, -1]
    offs, slot, src, dropped = R.plan(ids, 0, 3, 2, 6)
    assert offs.tolist() == [4, 4, 6] and dropped == 1 and slot.tolist() == [[4, 0], [5, -1], [-1, -1], [1, 2]] and src.tolist() == [1, 6, 7, -1, 0, 2]


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(3)
    ids = rng.integers(-1, 4, (5, 3))
    _, slot, src, _ = R.plan(ids, 0, 3, 4, 20)
    x, w, dout = rng.standard_normal((5, 6)), rng.standard_normal((5, 3)), rng.standard_normal((5, 6))
    scale = rng.standard_normal(20)  # what happens to a row between: the experts
    loss = lambda x, w: float((R.combine(R.dispatch(x, src, 3) * scale[:, None], w, slot)[0] * dout).sum())  # noqa: E731
    y = R.dispatch(x, src, 3) * scale[:, None]
    dy, dw, _ = R.combine_grad(dout, y, w, slot, 20)
    dx = R.combine(dy * scale[:, None], None, slot)[0]
    for at in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[at] = 1e-6
        assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-6 - dx[at]) < 1e-7
    for at in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[at] = 1e-6
        assert abs((loss(x, w + d) - loss(x, w - d)) / 2e-6 - dw[at]) < 1e-7
