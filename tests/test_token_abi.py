"""CPU tests of the C entry points of the layer norm and the gated delta rule:
bad arguments are refused with the documented status codes before anything is
enqueued, and calls without work succeed without a device."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "structured_state_space_dplr_amd", "libs4dplr.so")

OK, NULL, SHAPE, WORKSPACE, UNSUPPORTED, HIP, ALIAS, TOO_LARGE, ALIGN = range(9)
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from structured_state_space_dplr_amd.build import build
        build()
    import structured_state_space_dplr_amd as s4
    return s4._lib


def norm_fwd(lib, **kw):
    a = dict(x=MB, gamma=2 * MB, beta=3 * MB, y=4 * MB, mean=5 * MB, rstd=6 * MB, outer=4, D=32,
             inner=1, eps=1e-5, dtype=0)
    a.update(kw)
    return lib.s4dplr_layer_norm_fwd(*a.values(), None)


def norm_bwd(lib, **kw):
    a = dict(x=MB, gamma=2 * MB, mean=3 * MB, rstd=4 * MB, dy=5 * MB, dx=6 * MB, dgamma=7 * MB,
             dbeta=8 * MB, outer=4, D=32, inner=1, dtype=0, ws=9 * MB)
    a.update(kw)
    return lib.s4dplr_layer_norm_bwd(*a.values(), None)


def test_norm_sizes(lib):
    for bad in (dict(outer=-1), dict(D=0), dict(D=32769), dict(inner=0), dict(inner=1 << 31),
                dict(outer=1 << 31), dict(outer=1 << 20, inner=1 << 11),
                dict(outer=1 << 18, inner=1 << 10)):
        assert norm_fwd(lib, **bad) == SHAPE, bad
        assert norm_bwd(lib, **bad) == SHAPE, bad
    for eps in (-1e-9, float("nan"), float("inf")):
        assert norm_fwd(lib, eps=eps) == SHAPE
    for dtype in (-1, 3):
        assert norm_fwd(lib, dtype=dtype) == UNSUPPORTED
        assert norm_bwd(lib, dtype=dtype) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.s4dplr_layer_norm_workspace_bytes(4, 32, 1, None) == NULL
    assert lib.s4dplr_layer_norm_workspace_bytes(4, 0, 1, ctypes.byref(n)) == SHAPE
    assert lib.s4dplr_layer_norm_workspace_bytes(1 << 20, 1000, 1, ctypes.byref(n)) == OK
    assert n.value % 256 == 0 and 2 * 4 * 1000 <= n.value <= 64 * MB


def test_norm_pointers(lib):
    assert norm_fwd(lib, x=None) == NULL and norm_fwd(lib, y=None) == NULL
    for name in ("x", "mean", "rstd", "dy", "ws"):
        assert norm_bwd(lib, **{name: None}) == NULL
    assert norm_bwd(lib, ws=9 * MB + 8) == WORKSPACE
    for name in ("x", "gamma", "beta", "y", "mean", "rstd"):
        assert norm_fwd(lib, **{name: MB * 20 + 2}) == ALIGN, name
    for name in ("x", "gamma", "mean", "rstd", "dy", "dx", "dgamma", "dbeta"):
        assert norm_bwd(lib, **{name: MB * 20 + 2}) == ALIGN, name
    assert norm_fwd(lib, x=MB + 1, dtype=1) == ALIGN


def test_norm_overlaps(lib):
    size = 4 * 32 * 4
    for bad in (dict(y=MB + 4), dict(y=MB + size - 4), dict(mean=MB), dict(rstd=5 * MB),
                dict(y=2 * MB), dict(mean=4 * MB + size - 4)):
        assert norm_fwd(lib, **bad) == ALIAS, bad
    for bad in (dict(dx=5 * MB), dict(dx=MB), dict(dgamma=2 * MB), dict(dbeta=7 * MB),
                dict(dx=9 * MB), dict(dgamma=6 * MB)):
        assert norm_bwd(lib, **bad) == ALIAS, bad


def test_norm_without_work(lib):
    assert norm_fwd(lib, outer=0, x=None, y=None) == OK
    assert norm_bwd(lib, dx=None, dgamma=None, dbeta=None) == OK
    assert norm_bwd(lib, outer=0, dgamma=None, dbeta=None) == OK


def plan(lib, S=3, tokens=30, Hk=2, Hv=4, dk=16, dv=8, dtype=1, flags=0):
    h = ctypes.c_void_p()
    st = lib.s4dplr_delta_plan_create(ctypes.byref(h), S, tokens, Hk, Hv, dk, dv, dtype, flags)
    return st, h


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(tokens=0), OK), (dict(dk=256, dv=256, dtype=0, flags=1), OK),
    (dict(S=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(dk=0), SHAPE), (dict(dk=257), SHAPE), (dict(dv=0), SHAPE), (dict(dv=257), SHAPE),
    (dict(Hk=0), SHAPE), (dict(Hv=0), SHAPE), (dict(Hk=3), SHAPE), (dict(Hv=65536), SHAPE),
    (dict(S=1 << 23), SHAPE), (dict(S=(1 << 16) + 1), SHAPE), (dict(tokens=1 << 29), SHAPE),
    (dict(tokens=1 << 28, Hk=1, Hv=1), SHAPE), (dict(dtype=3), UNSUPPORTED), (dict(flags=2), UNSUPPORTED)])
def test_delta_plan(lib, kw, expect):
    st, h = plan(lib, **kw)
    assert st == expect
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    if st != OK:
        assert h.value is None
        return
    assert lib.s4dplr_delta_plan_bytes(h, ctypes.byref(a), ctypes.byref(b)) == OK
    assert a.value > 0 and a.value % 256 == 0
    assert (b.value > 0) == bool(kw.get("flags"))
    assert lib.s4dplr_delta_plan_bytes(h, ctypes.byref(a), None) == OK
    assert lib.s4dplr_delta_plan_bytes(h, None, None) == NULL
    lib.s4dplr_delta_plan_destroy(h)


def test_delta_plan_null(lib):
    assert lib.s4dplr_delta_plan_create(None, 1, 1, 1, 1, 1, 1, 1, 0) == NULL
    assert lib.s4dplr_delta_plan_bytes(None, None, None) == NULL
    lib.s4dplr_delta_plan_destroy(None)


G = 1 << 30
FWD = dict(q=G, ldq=32, k=2 * G, ldk=32, v=3 * G, ldv=32, g=4 * G, beta=5 * G, offsets=6 * G,
           scale=1.0, state=7 * G, o=8 * G, state_out=9 * G, saved=None, ws=10 * G)
BWD = dict(q=G, ldq=32, k=2 * G, ldk=32, v=3 * G, ldv=32, g=4 * G, beta=5 * G, offsets=6 * G,
           scale=1.0, saved=7 * G, dout=8 * G, dstate_out=9 * G, dq=10 * G, dk=11 * G, dv=12 * G,
           dg=13 * G, dbeta=14 * G, dstate=15 * G, ws=16 * G)


def delta(lib, h, base, **kw):
    fn = lib.s4dplr_delta_fwd if "o" in base else lib.s4dplr_delta_bwd
    return fn(h, *{**base, **kw}.values(), None)


def test_delta_pointers(lib):
    _, h = plan(lib)
    _, t = plan(lib, flags=1)
    for name in ("q", "k", "v", "g", "beta", "o", "ws"):
        assert delta(lib, h, FWD, **{name: None}) == NULL, name
    for name in ("q", "k", "v", "g", "beta", "dout", "saved", "ws"):
        assert delta(lib, t, BWD, **{name: None}) == NULL, name
    assert delta(lib, None, FWD) == NULL and delta(lib, None, BWD) == NULL
    assert delta(lib, h, FWD, saved=20 * G) == UNSUPPORTED
    assert delta(lib, h, BWD) == UNSUPPORTED
    assert delta(lib, h, FWD, ws=10 * G + 128) == WORKSPACE
    assert delta(lib, t, FWD, saved=20 * G + 64) == WORKSPACE
    assert delta(lib, t, BWD, saved=7 * G + 64) == WORKSPACE
    for name in ("q", "k", "v", "g", "beta", "offsets", "state", "o", "state_out"):
        assert delta(lib, h, FWD, **{name: FWD[name] + 1}) == ALIGN, name
    for name in ("dout", "dstate_out", "dq", "dk", "dv", "dg", "dbeta", "dstate"):
        assert delta(lib, t, BWD, **{name: BWD[name] + 1}) == ALIGN, name
    lib.s4dplr_delta_plan_destroy(h)
    lib.s4dplr_delta_plan_destroy(t)


def test_delta_sizes(lib):
    _, h = plan(lib, tokens=31)
    for name in ("ldq", "ldk", "ldv"):
        for bad in (31, -32, 1 << 31):
            assert delta(lib, h, FWD, **{name: bad}) == SHAPE, name
    assert delta(lib, h, FWD, offsets=None) == SHAPE      # 31 rows are no 3 equal sequences
    lib.s4dplr_delta_plan_destroy(h)


def test_delta_overlaps(lib):
    _, h = plan(lib)
    _, t = plan(lib, flags=1)
    rows = 2 * (29 * 32 + 32)
    for bad in (dict(o=3 * G), dict(o=G + rows - 2), dict(o=4 * G + 30 * 4 * 4 - 4), dict(o=9 * G),
                dict(state_out=7 * G + 4), dict(state_out=8 * G), dict(o=10 * G + 256),
                dict(o=6 * G + 12), dict(state_out=10 * G)):
        assert delta(lib, h, FWD, **bad) == ALIAS, bad
    assert delta(lib, t, FWD, saved=10 * G) == ALIAS
    # a wider pitch reaches further
    assert delta(lib, h, FWD, ldq=64, o=G + 2 * (29 * 64 + 30)) == ALIAS
    for bad in (dict(dq=G), dict(dk=8 * G), dict(dv=11 * G), dict(dg=14 * G), dict(dbeta=5 * G),
                dict(dstate=9 * G + 4), dict(dq=7 * G + 512), dict(dg=16 * G + 512)):
        assert delta(lib, t, BWD, **bad) == ALIAS, bad
    lib.s4dplr_delta_plan_destroy(h)
    lib.s4dplr_delta_plan_destroy(t)


def test_header_names_every_entry(lib):
    text = open(os.path.join(ROOT, "include", "s4dplr.h")).read()
    for n in ("layer_norm_fwd", "layer_norm_bwd", "layer_norm_workspace_bytes", "delta_plan_create",
              "delta_plan_bytes", "delta_plan_destroy", "delta_fwd", "delta_bwd"):
        assert f"s4dplr_{n}(" in text and hasattr(lib, f"s4dplr_{n}")


@pytest.mark.parametrize("at", range(6))
@pytest.mark.parametrize("size", [1 << 32, (1 << 32) + 1, -(1 << 32) + 1])
def test_plan_sizes_of_more_than_32_bits(lib, at, size):
    import structured_state_space_dplr_amd as s4
    sizes = [1, 64, 1, 1, 16, 16]
    sizes[at] = size
    with pytest.raises(s4.S4DPLRError) as e:
        s4.DeltaPlan(*sizes)
    assert e.value.status == SHAPE
