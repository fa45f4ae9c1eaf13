"""CPU tests of the C entry points of linear attention, the root-mean-square norm,
quantization to 8 bits and the 8-bit product: bad arguments are refused with the documented
status codes before anything is enqueued, and calls without work succeed without a device."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "structured_state_space_dplr_amd", "libs4dplr.so")

OK, NULL, SHAPE, WORKSPACE, UNSUPPORTED, HIP, ALIAS, TOO_LARGE, ALIGN = range(9)
MB, G = 1 << 20, 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from structured_state_space_dplr_amd.build import build
        build()
    import structured_state_space_dplr_amd as s4
    return s4._lib


def rms_fwd(lib, **kw):
    a = dict(x=MB, residual=2 * MB, gamma=3 * MB, h=4 * MB, y=5 * MB, q=6 * MB, scales=7 * MB, rstd=8 * MB, rows=4,
             D=300, eps=1e-5, dtype=0)
    a.update(kw)
    return lib.s4dplr_rms_norm_fwd(*a.values(), None)


def rms_bwd(lib, **kw):
    a = dict(h=MB, gamma=2 * MB, rstd=3 * MB, dy=4 * MB, dh=5 * MB, dx=6 * MB, dgamma=7 * MB, rows=4, D=300, dtype=0,
             ws=8 * MB)
    a.update(kw)
    return lib.s4dplr_rms_norm_bwd(*a.values(), None)


def test_rms_sizes(lib):
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(D=0), dict(D=32769)):
        assert rms_fwd(lib, **bad) == SHAPE and rms_bwd(lib, **bad) == SHAPE, bad
    for eps in (-1e-9, float("nan"), float("inf")):
        assert rms_fwd(lib, eps=eps) == SHAPE
    for dtype in (-1, 3):
        assert rms_fwd(lib, dtype=dtype) == UNSUPPORTED and rms_bwd(lib, dtype=dtype) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.s4dplr_rms_norm_workspace_bytes(4, 32, None) == NULL
    assert lib.s4dplr_rms_norm_workspace_bytes(4, 0, ctypes.byref(n)) == SHAPE
    assert lib.s4dplr_rms_norm_workspace_bytes(1 << 20, 1000, ctypes.byref(n)) == OK
    assert n.value % 256 == 0 and 4000 <= n.value <= 32 * MB


def test_rms_pointers(lib):
    assert rms_fwd(lib, x=None) == NULL and rms_fwd(lib, q=None) == NULL and rms_fwd(lib, scales=None) == NULL
    assert rms_fwd(lib, y=None, q=None, scales=None) == NULL
    for name in ("h", "rstd", "dy", "ws"):
        assert rms_bwd(lib, **{name: None}) == NULL, name
    assert rms_bwd(lib, ws=8 * MB + 8) == WORKSPACE
    for name in ("x", "residual", "gamma", "h", "y", "rstd"):
        assert rms_fwd(lib, **{name: 20 * MB + 2}) == ALIGN, name
    for name in ("h", "gamma", "rstd", "dy", "dh", "dx", "dgamma"):
        assert rms_bwd(lib, **{name: 20 * MB + 2}) == ALIGN, name


def test_rms_overlaps(lib):
    size = 4 * 300 * 4
    for bad in (dict(h=MB), dict(h=2 * MB + 4), dict(y=2 * MB), dict(y=4 * MB + size - 4), dict(q=MB + size - 1),
                dict(scales=6 * MB + 1199), dict(rstd=5 * MB), dict(y=MB)):
        assert rms_fwd(lib, **bad) == ALIAS, bad
    for bad in (dict(dx=4 * MB), dict(dx=5 * MB + 4), dict(dgamma=2 * MB), dict(dx=8 * MB), dict(dgamma=6 * MB)):
        assert rms_bwd(lib, **bad) == ALIAS, bad


def test_rms_without_work(lib):
    assert rms_fwd(lib, rows=0, x=None, y=None, q=None, scales=None) == OK
    assert rms_bwd(lib, dx=None, dgamma=None) == OK
    assert rms_bwd(lib, rows=0, dgamma=None) == OK


def quantize(lib, **kw):
    a = dict(x=MB, ldx=300, q=2 * MB, scales=3 * MB, qt=4 * MB, scales_t=5 * MB, rows=200, cols=300, square=0, dtype=1)
    a.update(kw)
    return lib.s4dplr_quantize_fp8(*a.values(), None)


def test_quantize(lib):
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=(1 << 22) + 1), dict(cols=1 << 24), dict(ldx=299),
                dict(ldx=1 << 24), dict(rows=1 << 22, cols=1 << 16, ldx=1 << 16)):
        assert quantize(lib, **bad) == SHAPE, bad
    assert quantize(lib, dtype=3) == UNSUPPORTED
    for name in ("x", "q", "scales", "qt", "scales_t"):
        assert quantize(lib, **{name: None}) == NULL, name
    assert quantize(lib, x=MB + 1) == ALIGN
    for bad in (dict(q=MB), dict(q=MB + 200 * 300 * 2 - 1), dict(scales=2 * MB + 59999), dict(qt=2 * MB),
                dict(scales_t=4 * MB + 1), dict(scales=MB + 5), dict(q=3 * MB + 599)):
        assert quantize(lib, **bad) == ALIAS, bad
    assert quantize(lib, rows=0) == OK and quantize(lib, cols=0) == OK
    assert quantize(lib, q=None, scales=None, qt=None, scales_t=None) == OK


def matmul(lib, **kw):
    a = dict(a=MB, lda=300, sa=2 * MB, b=3 * MB, ldb=300, sb=4 * MB, square=0, out=5 * MB, ldo=70, M=50, N=70, K=300,
             dtype=1)
    a.update(kw)
    return lib.s4dplr_matmul_fp8(*a.values(), None)


def test_matmul(lib):
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 24), dict(lda=299), dict(ldb=299), dict(ldo=69),
                dict(lda=1 << 24), dict(ldo=1 << 24), dict(M=1 << 23, N=1 << 20, ldo=1 << 20)):
        assert matmul(lib, **bad) == SHAPE, bad
    assert matmul(lib, dtype=-1) == UNSUPPORTED
    for name in ("a", "sa", "b", "sb", "out"):
        assert matmul(lib, **{name: None}) == NULL, name
    assert matmul(lib, out=5 * MB + 1) == ALIGN
    for bad in (dict(out=MB), dict(out=2 * MB), dict(out=3 * MB + 300 * 70 - 2), dict(out=4 * MB + 208)):
        assert matmul(lib, **bad) == ALIAS, bad
    assert matmul(lib, M=0) == OK and matmul(lib, N=0) == OK


def plan(lib, S=3, tokens=30, Hk=2, Hv=4, dk=16, dv=8, dtype=1, flags=0):
    h = ctypes.c_void_p()
    st = lib.s4dplr_linear_attention_plan_create(ctypes.byref(h), S, tokens, Hk, Hv, dk, dv, dtype, flags)
    return st, h


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK), (dict(tokens=0), OK), (dict(dk=256, dv=256, dtype=0, flags=1), OK),
    (dict(S=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(dk=0), SHAPE), (dict(dk=257), SHAPE), (dict(dv=0), SHAPE), (dict(dv=257), SHAPE),
    (dict(Hk=0), SHAPE), (dict(Hv=0), SHAPE), (dict(Hk=3), SHAPE), (dict(Hv=65536), SHAPE),
    (dict(S=1 << 23), SHAPE), (dict(S=(1 << 16) + 1), SHAPE), (dict(tokens=1 << 29), SHAPE),
    (dict(dtype=3), UNSUPPORTED), (dict(flags=2), UNSUPPORTED)])
def test_linear_plan(lib, kw, expect):
    st, h = plan(lib, **kw)
    assert st == expect
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    if st != OK:
        assert h.value is None
        return
    assert lib.s4dplr_linear_attention_plan_bytes(h, ctypes.byref(a), ctypes.byref(b)) == OK
    assert a.value > 0 and a.value % 256 == 0 and (b.value > 0) == bool(kw.get("flags"))
    assert lib.s4dplr_linear_attention_plan_bytes(h, ctypes.byref(a), None) == OK
    assert lib.s4dplr_linear_attention_plan_bytes(h, None, None) == NULL
    lib.s4dplr_linear_attention_plan_destroy(h)


def test_linear_plan_null(lib):
    assert lib.s4dplr_linear_attention_plan_create(None, 1, 1, 1, 1, 1, 1, 1, 0) == NULL
    assert lib.s4dplr_linear_attention_plan_bytes(None, None, None) == NULL
    lib.s4dplr_linear_attention_plan_destroy(None)


@pytest.mark.parametrize("sequences,tokens,most", [(1, 1, 1 << 10), (128, 128, 4 << 20), (16384, 16384, 64 << 20),
                                                   (1, 16384, 64 << 20), (4, 16384, 64 << 20)])
def test_linear_workspace(sequences, tokens, most):
    """States between segments alone, as many as there can be (16 value heads of 128 x 128, a
    megabyte each): three for 128 tokens, which may be one sequence."""
    import structured_state_space_dplr_amd as s4
    p = s4.LinearAttentionPlan(sequences, tokens, 8, 16, 128, 128, device="cpu")
    assert 0 < p.workspace_bytes <= most


@pytest.mark.parametrize("at", range(6))
@pytest.mark.parametrize("size", [1 << 32, (1 << 32) + 1, -(1 << 32) + 1])
def test_plan_sizes_of_more_than_32_bits(lib, at, size):
    import structured_state_space_dplr_amd as s4
    sizes = [1, 64, 1, 1, 16, 16]
    sizes[at] = size
    with pytest.raises(s4.S4DPLRError) as e:
        s4.LinearAttentionPlan(*sizes)
    assert e.value.status == SHAPE


FWD = dict(q=G, ldq=32, k=2 * G, ldk=32, v=3 * G, ldv=32, g=4 * G, fixed=0, offsets=6 * G, scale=1.0, state=7 * G,
           o=8 * G, state_out=9 * G, saved=None, ws=10 * G)
BWD = dict(q=G, ldq=32, k=2 * G, ldk=32, v=3 * G, ldv=32, g=4 * G, fixed=0, offsets=6 * G, scale=1.0, saved=7 * G,
           dout=8 * G, dstate_out=9 * G, dq=10 * G, dk=11 * G, dv=12 * G, dg=13 * G, dstate=15 * G, ws=16 * G)


def linear(lib, h, base, **kw):
    fn = lib.s4dplr_linear_attention_fwd if "o" in base else lib.s4dplr_linear_attention_bwd
    return fn(h, *{**base, **kw}.values(), None)


def test_linear_pointers(lib):
    _, h = plan(lib)
    _, t = plan(lib, flags=1)
    for name in ("q", "k", "v", "o", "ws"):
        assert linear(lib, h, FWD, **{name: None}) == NULL, name
    for name in ("q", "k", "v", "g", "dout", "saved", "ws"):
        assert linear(lib, t, BWD, **{name: None}) == NULL, name
    assert linear(lib, None, FWD) == NULL and linear(lib, None, BWD) == NULL
    assert linear(lib, h, FWD, saved=20 * G) == UNSUPPORTED and linear(lib, h, BWD) == UNSUPPORTED
    assert linear(lib, h, FWD, ws=10 * G + 128) == WORKSPACE
    assert linear(lib, t, FWD, saved=20 * G + 64) == WORKSPACE
    assert linear(lib, t, BWD, saved=7 * G + 64) == WORKSPACE
    for name in ("q", "k", "v", "g", "offsets", "state", "o", "state_out"):
        assert linear(lib, h, FWD, **{name: FWD[name] + 1}) == ALIGN, name
    for name in ("dout", "dstate_out", "dq", "dk", "dv", "dg", "dstate"):
        assert linear(lib, t, BWD, **{name: BWD[name] + 1}) == ALIGN, name
    lib.s4dplr_linear_attention_plan_destroy(h)
    lib.s4dplr_linear_attention_plan_destroy(t)


def test_linear_sizes_and_overlaps(lib):
    _, h = plan(lib, tokens=31)
    for name in ("ldq", "ldk", "ldv"):
        for bad in (31, -32, 1 << 31):
            assert linear(lib, h, FWD, **{name: bad}) == SHAPE, name
    assert linear(lib, h, FWD, offsets=None) == SHAPE      # 31 rows are no 3 equal sequences
    lib.s4dplr_linear_attention_plan_destroy(h)
    _, h = plan(lib)
    _, t = plan(lib, flags=1)
    rows = 2 * (29 * 32 + 32)
    for bad in (dict(o=3 * G), dict(o=G + rows - 2), dict(o=4 * G + 30 * 4 * 4 - 4), dict(o=9 * G),
                dict(state_out=7 * G + 4), dict(state_out=8 * G), dict(o=10 * G), dict(o=6 * G + 12),
                dict(state_out=10 * G)):
        assert linear(lib, h, FWD, **bad) == ALIAS, bad
    assert linear(lib, h, FWD, fixed=1, o=4 * G + 12) == ALIAS
    assert linear(lib, t, FWD, saved=10 * G) == ALIAS
    for bad in (dict(dq=G), dict(dk=8 * G), dict(dv=11 * G), dict(dg=4 * G), dict(dstate=9 * G + 4),
                dict(dq=7 * G + 512), dict(dg=16 * G + 512)):
        assert linear(lib, t, BWD, **bad) == ALIAS, bad
    lib.s4dplr_linear_attention_plan_destroy(h)
    lib.s4dplr_linear_attention_plan_destroy(t)


def test_header_names_every_entry(lib):
    text = open(os.path.join(ROOT, "include", "s4dplr.h")).read()
    for n in ("linear_attention_plan_create", "linear_attention_plan_bytes", "linear_attention_plan_destroy",
              "linear_attention_fwd", "linear_attention_bwd", "rms_norm_fwd", "rms_norm_bwd",
              "rms_norm_workspace_bytes", "quantize_fp8", "matmul_fp8"):
        assert f"s4dplr_{n}(" in text and hasattr(lib, f"s4dplr_{n}")
