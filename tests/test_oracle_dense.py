"""The dense operators' oracle against exact integer sums, a row quantised by hand and
torch's own activation, and the argument checks of their entry points (which return before
any HIP call, so they run without a GPU)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mixture_experts_layer_route_amd as moe
from oracle import dense as od

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_quant_i8_by_hand():
    v = np.array([[0.0, 0.5, -1.27, 0.015, -0.025, 0.005], [0, 0, 0, 0, 0, 0]])
    codes, scale = od.quant_i8(v)
    np.testing.assert_allclose(scale, [0.01, 1.0], rtol=1e-15)
    assert codes[0].tolist()[:3] == [0, 50, -127]
    assert (codes[1] == 0).all()
    assert np.abs(codes * scale[:, None] - v).max() <= 0.005 * (1 + 1e-12)


def test_product_against_python_integers():
    rng = np.random.default_rng(3)
    x = rng.integers(-128, 128, (3, 48))
    w = rng.integers(-128, 128, (5, 48))
    x[0], w[0] = -128, -128                       # the largest sum a row can have
    sx, sw = rng.random(3) + 0.5, rng.random(5) + 0.5
    got = od.product(x, sx, w, sw)
    for t in range(3):
        for n in range(5):
            acc = sum(int(a) * int(b) for a, b in zip(x[t], w[n]))
            assert got[t, n] == pytest.approx(acc * sx[t] * sw[n], rel=1e-15)


def test_glu_against_torch():
    rng = np.random.default_rng(4)
    x, wg, wu = (rng.integers(-127, 128, s) for s in ((4, 32), (6, 32), (6, 32)))
    one4, one6 = np.full(4, 0.01), np.full(6, 0.02)
    g, u = (torch.from_numpy(od.product(x, one4, w, one6)) for w in (wg, wu))
    want = torch.nn.functional.silu(g) * u
    np.testing.assert_allclose(od.glu(x, one4, wg, one6, wu, one6), want.numpy(), rtol=1e-12)


def test_norm_against_torch_and_sum_rounding():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((3, 64))).to(torch.bfloat16)
    r = torch.from_numpy(rng.standard_normal((3, 64))).to(torch.bfloat16)
    gamma = rng.standard_normal(64)
    s = od.summed_rows(x.double().numpy(), r.double().numpy())
    assert np.array_equal(s, (x + r).double().numpy())
    want = torch.nn.functional.rms_norm((x + r).double(), (64,), torch.from_numpy(gamma), 1e-6)
    np.testing.assert_allclose(od.norm_rows(x.double().numpy(), gamma, r.double().numpy()),
                               want.numpy(), rtol=1e-12)


# ------------------------------------------------------------------ argument checks

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return moe.load_library()


FAKE = 1 << 40          # never dereferenced: validation fails first
ROWS = dict(rows=4, width=1536, act=1, fmt=1, x=FAKE, res=None, gamma=FAKE, eps=1e-6, x_sum=None,
            out=FAKE, scales=FAKE)
PROD = dict(rows=4, K=1536, N=512, out=1, x=FAKE, sx=FAKE, w=FAKE, sw=FAKE, res=None, y=FAKE)
GLU = dict(rows=4, K=1536, N=512, out=1, x=FAKE, sx=FAKE, w=FAKE, sw=FAKE, wu=FAKE, su=FAKE, y=FAKE)


def _call(fn, base, **kw):
    return fn(*({**base, **kw}.values()), None)


@pytest.mark.parametrize("code,kw", [
    (-1, dict(rows=0)), (-1, dict(rows=-3)), (-1, dict(width=0)), (-1, dict(x=None)),
    (-1, dict(out=None)), (-1, dict(scales=None)), (-1, dict(res=FAKE)),   # a residual without x_sum
    (-1, dict(eps=-1.0)), (-1, dict(eps=float("nan"))), (-1, dict(x=FAKE + 8)),
    (-1, dict(gamma=FAKE + 2)), (-1, dict(out=FAKE + 4)), (-1, dict(res=FAKE + 8, x_sum=FAKE)),
    (-1, dict(res=FAKE, x_sum=FAKE + 8)), (-1, dict(scales=FAKE + 2)),
    (-2, dict(act=2)), (-2, dict(act=-1)), (-2, dict(fmt=4)), (-2, dict(fmt=-1)),
    (-2, dict(width=1532)), (-2, dict(fmt=2, width=1600)), (-2, dict(fmt=3, width=1544)),
    (-2, dict(width=32776)), (-2, dict(rows=(1 << 21) + 1)), (-2, dict(rows=1 << 40)),
])
def test_norm_quant_rows_refuses(lib, code, kw):
    assert _call(lib.moe_norm_quant_rows, ROWS, **kw) == code


BAD_PRODUCT = [
    (-1, dict(rows=0)), (-1, dict(K=0)), (-1, dict(N=0)), (-1, dict(x=None)), (-1, dict(sx=None)),
    (-1, dict(w=None)), (-1, dict(sw=None)), (-1, dict(y=None)), (-1, dict(x=FAKE + 8)),
    (-1, dict(w=FAKE + 1)), (-1, dict(sx=FAKE + 2)), (-1, dict(sw=FAKE + 1)), (-1, dict(y=FAKE + 1)),
    (-1, dict(out=0, y=FAKE + 2)), (-2, dict(out=2)), (-2, dict(K=1544)), (-2, dict(K=65552)),
    (-2, dict(rows=(1 << 21) + 1)), (-2, dict(rows=1 << 40)), (-2, dict(N=(1 << 24) + 1)),
    (-2, dict(rows=1 << 21, N=(1 << 14) + 1)),
]


@pytest.mark.parametrize("code,kw", BAD_PRODUCT + [(-1, dict(res=FAKE + 1))])
def test_linear_i8_refuses(lib, code, kw):
    assert _call(lib.moe_linear_i8, PROD, **kw) == code


@pytest.mark.parametrize("code,kw", BAD_PRODUCT + [(-1, dict(wu=None)), (-1, dict(su=None)),
                                                   (-1, dict(wu=FAKE + 8)), (-1, dict(su=FAKE + 2))])
def test_glu_i8_refuses(lib, code, kw):
    assert _call(lib.moe_glu_i8, GLU, **kw) == code


def test_dense_layer_refuses(lib):
    n = ctypes.c_size_t(0)
    size = lib.moe_dense_workspace_size
    cfg = lambda *a: ctypes.byref(moe.make_dense_config(*a))
    for code, args in ((-1, (0, 1536, 512)), (-1, (4, 0, 512)), (-1, (4, 1536, 0)), (-2, (4, 1528, 512)),
                       (-2, (4, 1536, 520)), (-2, (4, 1536, 512, "e4m3")), (-2, (4, 32784, 512)),
                       (-2, (4, 1536, 32784)), (-2, ((1 << 21) + 1, 1536, 512)), (-2, (1 << 21, 512, 16400))):
        assert size(cfg(*args), ctypes.byref(n)) == code, args
    assert size(None, ctypes.byref(n)) == -1 and size(cfg(4, 1536, 512), None) == -1
    assert size(cfg(4, 1536, 512), ctypes.byref(n)) == 0 and n.value > 0
    full = moe.DenseWeights(*[FAKE] * 6)
    run = lambda c=cfg(4, 1536, 512), x=FAKE, g=FAKE, eps=1e-6, w=full, o=FAKE, ws=FAKE, b=n.value: \
        lib.moe_dense_residual_i8(c, x, g, eps, ctypes.byref(w) if w is not None else None, o, ws, b, None)
    assert run(x=None) == run(g=None) == run(o=None) == run(ws=None) == run(w=None) == run(c=None) == -1
    assert run(eps=-1.0) == run(eps=float("nan")) == run(ws=FAKE + 16) == -1
    assert run(x=FAKE + 8) == run(g=FAKE + 8) == run(o=FAKE + 1) == run(o=FAKE + 8) == -1
    assert run(b=n.value - 1) == -3
    for i in range(6):
        assert run(w=moe.DenseWeights(*[None if j == i else FAKE for j in range(6)])) == -1, i


def test_dense_structs_match_header():
    txt = open(os.path.join(ROOT, "include", "moe.h")).read()
    for name, st in (("moe_dense_config", moe.DenseConfig), ("moe_dense_weights", moe.DenseWeights)):
        end = txt.index("} %s;" % name)
        body = txt[txt.rindex("typedef struct {", 0, end):end]
        assert re.findall(r"^\s*(?:const )?\w+\*?\s+(\w+);", body, re.M) == [n for n, _ in st._fields_]


def test_binding_refuses_before_the_library():
    i8 = torch.zeros((2, 32), dtype=torch.int8)
    f = torch.ones(2)
    with pytest.raises(ValueError, match="current device"):
        moe.linear_i8(i8, f, i8, f)                              # host tensors
    with pytest.raises(ValueError, match="x_codes"):
        moe.linear_i8(i8.float(), f, i8, f)
    with pytest.raises(ValueError, match="out_dtype"):
        moe.linear_i8(i8, f, i8, f, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="rows, width"):
        moe.norm_quant_rows(f, "i8")
    with pytest.raises(ValueError, match="fmt"):
        moe.norm_quant_rows(torch.zeros(2, 32), "int8")
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        moe.norm_quant_rows(torch.zeros((2, 32), dtype=torch.float16), "i8")
