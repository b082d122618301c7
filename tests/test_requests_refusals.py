"""Calls of the many-adapter operators that the host refuses (CPU): outputs that
overlap an input, another output or the workspace.  Every call here is refused,
so none reaches a device, whatever the machine has."""
import ctypes

import pytest

OVERLAP = 10


@pytest.fixture(scope="module")
def q4():
    import parameter_efficient_fine_nf4_b200 as q4
    from parameter_efficient_fine_nf4_b200 import build
    build.build()
    return q4


K, D, ROWS, WIDTH, T = 256, 512, 64, 32, 100
SIZES = dict(A=ROWS * K * 2, Bt=ROWS * D * 2, X=T * K * 2, Y=T * D * 2, base_y=T * D * 2, U=T * WIDTH * 4, dY=T * D * 2,
             dX=T * K * 2, base_x=T * K * 2, dA=ROWS * K * 4, dBt=ROWS * D * 4)
SIZE_WS = 1 << 22


def _layout():
    """Disjoint addresses with 16 bytes between them."""
    at, out = 1 << 20, {}
    for name, size in list(SIZES.items()) + [("ws", SIZE_WS)]:
        out[name] = at
        at += size + 16
    return out


def _structs(q4, a):
    pool = q4._Pool(a["A"], a["Bt"], 16, 16, 16, ROWS, K, D, 3, WIDTH)
    return pool, q4._Requests(16, 16, 16, 16, 16, 16, T, 2, 3)


def _fwd(q4, a, layer):
    pool, req = _structs(q4, a)
    L, P, R = q4.lib(), ctypes.byref(pool), ctypes.byref(req)
    if layer:
        nf4 = ctypes.byref(q4._NF4(16, 16, 16, 16, D, K, 64, 256))
        return L.qlora_fwd_requests(nf4, P, R, a["X"], a["Y"], a["U"], a["ws"], SIZE_WS, None)
    return L.lora_requests_fwd(P, R, a["X"], a["base_y"], a["Y"], a["U"], a["ws"], SIZE_WS, None)


def _bwd(q4, a, layer):
    pool, req = _structs(q4, a)
    L, P, R = q4.lib(), ctypes.byref(pool), ctypes.byref(req)
    if layer:
        nf4 = ctypes.byref(q4._NF4(16, 16, 16, 16, D, K, 64, 256))
        return L.qlora_bwd_requests(nf4, P, R, a["X"], a["U"], a["dY"], a["dX"], a["dA"], a["dBt"], a["ws"], SIZE_WS, None)
    return L.lora_requests_bwd(P, R, a["X"], a["U"], a["dY"], a["base_x"], a["dX"], a["dA"], a["dBt"], a["ws"], SIZE_WS,
                               None)


FWD = [(o, i) for o in ("Y", "U", "ws") for i in ("X", "A", "Bt", "base_y")] + [("Y", "U"), ("Y", "ws"), ("U", "ws")]
BWD = [(o, i) for o in ("dX", "dA", "dBt", "ws") for i in ("X", "U", "dY", "A", "Bt", "base_x")] + [
    ("dX", "dA"), ("dX", "dBt"), ("dX", "ws"), ("dA", "dBt"), ("dA", "ws"), ("dBt", "ws")]


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("call,pairs", [("fwd", FWD), ("bwd", BWD)])
def test_overlaps_are_refused(q4, call, pairs, layer):
    run = _fwd if call == "fwd" else _bwd
    sizes = dict(SIZES, ws=256)                  # the least that any workspace has
    for x, y in pairs:
        if layer and "base" in y:
            continue
        for first, second in ((x, y), (y, x)):   # the last 16 bytes of one, the first of the other
            a = _layout()
            a[second] = a[first] + sizes[first] - 16
            assert run(q4, a, layer) == OVERLAP, (x, y, first)


def test_equal_addresses(q4):
    for layer in (False, True):
        a = _layout()
        assert _fwd(q4, dict(a, Y=a["X"]), layer) == 1
        assert _bwd(q4, dict(a, dX=a["X"]), layer) == 1
        assert _bwd(q4, dict(a, dX=a["dY"]), layer) == 1
        assert _fwd(q4, dict(a, U=a["Y"]), layer) == OVERLAP
        assert _bwd(q4, dict(a, dBt=a["dA"]), layer) == OVERLAP
        assert _bwd(q4, dict(a, dX=a["U"]), layer) == OVERLAP
    assert q4.strerror(OVERLAP) == "an output overlaps another argument"


@pytest.mark.parametrize("coefs,most", [(None, 8), ((3.4445, -4.7750, 2.0315), 8), ((4.0848, -6.8946, 2.9270), 7),
                                        ((-4.0848, 6.0, -2.0), 7), ((3.0, -3.2, 1.2), 9), ((2.0, -1.5, 0.5), 15),
                                        ((0.5, 0.6, -0.1), 16)])
def test_steps_that_the_gram_matrix_does_not_hold(q4, coefs, most):
    """|a|^(2 steps) <= 2^30, and 16 at most; the steps that pass are refused for their workspace (4)."""
    cs = None if coefs is None else (ctypes.c_float * 3)(*coefs)
    for steps in range(1, 20):
        got = q4.lib().lora_muon_step(16, 16, 16, 16, 1, 16, 256, 0.1, 0.9, 1, 1.0, 0.0, 1e-7, steps,
                                      None if cs is None else ctypes.addressof(cs), 16, 16, None)
        assert got == (4 if steps <= most else 1), steps
