"""GPU parity of the dense 8-bit operators against the float64 oracle.

Bounds, with u = 2^-24 (half an ulp of fp32, relative) and e = eps / 2 of the output type:
  * product: the sum is exact; its conversion to fp32 and two multiplications cost 3 u of the
    product, the residual's addition u of the result, the store e of the result.
  * norm: the squares are summed in chains of at most 32 fused steps per lane and 22 additions
    across lanes (relative error of a sum of non-negative terms <= the longest chain), halved by
    the root: 27 u; mean, eps, root, reciprocal and two products add 6 u.  33 u, taken as 40 u.
  * codes: the quotient v / scale (1 u more, and the scale's own 41 u enters both sides of the
    comparison, which uses the stored scale) is rounded to the grid: half a grid step plus
    42 u of the quotient.
  * gated product: g and u carry 3 u each; an error d of g changes silu by at most (1 + |g|) d
    relative, exp's argument rounding adds 2 |g| u, exp, sum, quotient and products 6 u:
    (12 + 6 |g|) u.  Where exp(-g) overflows (g < -88) the result is 0 instead of < 1e-36 |u|.
  * dense layer: see layer_and_bound.
"""
import numpy as np
import pytest
import torch

from oracle import dense as od
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NORM = 40 * U
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_layer_route_amd as m
    m.load_library()
    return m


def f64(t):
    return t.double().cpu().numpy()


def store(dt):
    return torch.finfo(dt).eps / 2


def codes_of(g, rows, width):
    c = (torch.randn(rows, width, generator=g, device="cuda") * 40).round().clamp(-128, 127)
    return c.to(torch.int8), torch.rand(rows, generator=g, device="cuda") * 0.02 + 1e-3


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ norm + quantisation

def check_rows(out, scales, fmt, v, dt):
    """Stored rows or codes against the oracle's values v."""
    T, H = v.shape
    if fmt == "rows":
        assert (np.abs(f64(out) - v) <= (NORM + store(dt)) * np.abs(v) * (1 + 1e-6) + 1e-38).all()
        return
    n = {"i8": H, "e4m3": 128, "mxfp8": 32}[fmt]
    b = v.reshape(T, -1, n)
    amax = np.abs(b).max(axis=2)
    if fmt == "mxfp8":
        X = scales.cpu().numpy().astype(np.int64).reshape(T, -1) - 127
        lo, hi = (np.where(amax > 0, np.frexp(np.maximum(amax * f, 1e-300))[1] - 9, -127)
                  for f in (1 - NORM, 1 + NORM))
        assert ((X >= np.clip(lo, -127, 127)) & (X <= np.clip(hi, -127, 127))).all()
        s = np.exp2(X.astype(np.float64))
    else:
        s = f64(scales).reshape(T, -1)
        want = np.where(amax > 0, amax / {"i8": 127.0, "e4m3": 448.0}[fmt], 1.0)
        assert (np.abs(s - want) <= (NORM + 2 * U) * want).all()
    q = b / s[:, :, None]
    if fmt == "i8":
        c = out.cpu().numpy().astype(np.float64).reshape(b.shape)
        assert np.abs(c).max() <= 127
        step = 1.0
    else:
        c = mo.e4m3_decode(out.cpu().numpy()).reshape(b.shape)
        q = np.clip(q, -448, 448)
        # the grid's step at the larger of code and value
        e = np.maximum(np.frexp(np.maximum(np.abs(q), np.abs(c)))[1] - 1, -6)
        step = np.exp2(e - 3.0)
    assert (np.abs(c - q) <= step / 2 + (NORM + 2 * U) * np.abs(q)).all()


WIDTHS = {"rows": (8, 40, 512, 1000, 1536, 2056, 4096, 8200, 32768),
          "i8": (8, 40, 512, 1000, 1536, 2056, 4096, 8200, 32768),
          "e4m3": (128, 384, 1536, 2176, 8320, 32768), "mxfp8": (32, 1184, 1536, 2080, 8224, 32768)}


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", list(WIDTHS))
def test_norm_quant_rows(moe, fmt, act):
    dt = DT[act]
    for H in WIDTHS[fmt]:
        for T, res, norm in ((1, True, True), (5, False, True), (3, True, False), (7, False, False)):
            print("case: norm", fmt, act, T, H, res, norm, flush=True)
            g = gen(H + T)
            x = (torch.randn(T, H, generator=g, device="cuda") * 3).to(dt)
            r = torch.randn(T, H, generator=g, device="cuda").to(dt) if res else None
            w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dt) if norm else None
            out, scales, total = moe.norm_quant_rows(x, fmt, w, r, EPS)
            s = od.summed_rows(f64(x), f64(r) if res else None, act)
            if res:
                assert np.array_equal(f64(total), s)
            else:
                assert total is None
            check_rows(out, scales, fmt, s if w is None else mo.rms_norm(s, f64(w), EPS), dt)


@pytest.mark.parametrize("fmt,H", [("rows", 1536), ("i8", 1000), ("i8", 2048), ("e4m3", 512),
                                   ("e4m3", 1536), ("mxfp8", 1024), ("mxfp8", 2016), ("i8", 4112)])
def test_norm_batches(moe, fmt, H):
    """The one-wave-per-row batch kernels, with a ragged last workgroup."""
    T = 2051
    print("case: norm batch", fmt, T, H, flush=True)
    g = gen(H)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    out, scales, total = moe.norm_quant_rows(x, fmt, w, r, EPS)
    s = od.summed_rows(f64(x), f64(r))
    assert np.array_equal(f64(total), s)
    check_rows(out, scales, fmt, mo.rms_norm(s, f64(w), EPS), torch.bfloat16)


@pytest.mark.parametrize("fmt", ["i8", "e4m3", "mxfp8"])
def test_norm_zero_tiny_and_huge_rows(moe, fmt):
    """A zero row, zero blocks in a row, one value per row, values at the ends of the range."""
    H = 1536
    x = torch.zeros(6, H, device="cuda")
    x[1, 700] = -2.0
    x[2] = 1e-38
    x[3, ::7] = 1e37
    x[4] = 1.0
    x[5, 128:256] = torch.linspace(-3, 3, 128, device="cuda")
    out, scales, _ = moe.norm_quant_rows(x, fmt)
    v = f64(x)
    live = [0, 1, 3, 4, 5]                   # 1e-38 / 127 is no normal number: scale 1, code 0
    check_rows(out[live], scales[live], fmt, v[live], torch.float32)
    if fmt != "mxfp8":
        assert (scales[2] == 1).all() and (out[2] == 0).all()
    w = torch.ones(H, device="cuda")
    out, scales, _ = moe.norm_quant_rows(x[:2].contiguous(), fmt, w)
    check_rows(out, scales, fmt, mo.rms_norm(v[:2], np.ones(H), EPS), torch.float32)
    # without eps a zero row stays zero, the others are normalised as ever
    out, scales, _ = moe.norm_quant_rows(x[:2].contiguous(), fmt, w, eps=0.0)
    check_rows(out, scales, fmt, np.stack([v[0], mo.rms_norm(v[1], np.ones(H), 0.0)]), torch.float32)


@pytest.mark.parametrize("T,H", [(7, 512), (7, 2048), (2050, 1024), (5, 8192), (3, 16384)])
@pytest.mark.parametrize("fmt", list(WIDTHS))
def test_norm_rows_that_are_not_finite(moe, fmt, T, H):
    """A NaN, an infinity, a NaN in the residual: the row's scale (with the norm every block's, for
    an infinity at least its own block's) is not finite; the other rows keep their bits."""
    print("case: not finite", fmt, T, H, flush=True)
    g = gen(H)
    x, r = torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")
    gamma = torch.ones(H, device="cuda")
    bx, br = x.clone(), r.clone()
    bx[0, 5], bx[1, H - 1], br[2, H // 2] = float("nan"), float("inf"), float("nan")
    n = {"rows": 1, "i8": H, "e4m3": 128, "mxfp8": 32}[fmt]
    for w, hit in ((gamma, (True, False, True)), (None, (False, False, False))):
        out, sc, _ = moe.norm_quant_rows(x, fmt, w, r)
        bad, bsc, _ = moe.norm_quant_rows(bx, fmt, w, br)
        assert torch.equal(out[3:], bad[3:]) and (sc is None or torch.equal(sc[3:], bsc[3:]))
        if fmt == "rows":
            lost = ~torch.isfinite(bad[:3])
        elif fmt == "mxfp8":
            lost = bsc[:3] == 255
        else:
            lost = ~torch.isfinite(bsc[:3].reshape(3, -1))
        for t, at in enumerate((5, H - 1, H // 2)):
            assert lost[t, at // n]
            assert not hit[t] or lost[t].all()
            assert w is not None or lost[t].sum() == 1
    # quantised alone, zeros beside one infinity: nothing else is touched
    z = torch.zeros(T, H, device="cuda")
    z[1, 0] = float("-inf")
    out, sc, _ = moe.norm_quant_rows(z, fmt)
    assert (out[0].float() == 0).all() and (out[2:].float() == 0).all()


def test_norm_in_place_and_neighbours(moe):
    """x_sum may be x or the residual and a rows output x; nothing behind the rows changes."""
    T, H = 9, 1544
    g = gen(2)
    for act in ("bf16", "f32"):
        dt = DT[act]
        x = torch.randn(T, H, generator=g, device="cuda").to(dt)
        r = torch.randn(T, H, generator=g, device="cuda").to(dt)
        w = torch.rand(H, generator=g, device="cuda").to(dt)
        out, scales, total = moe.norm_quant_rows(x, "i8", w, r)
        for which in (0, 1):
            a, b = x.clone(), r.clone()
            o2, s2, t2 = moe.norm_quant_rows(a, "i8", w, b, x_sum=(a, b)[which])
            assert torch.equal(o2, out) and torch.equal(s2, scales) and torch.equal(t2, total)
            assert torch.equal((b, a)[which], (r, x)[which])
        rows, _, _ = moe.norm_quant_rows(x, "rows", w)
        a = x.clone()
        moe.norm_quant_rows(a, "rows", w, out=a)
        assert torch.equal(a, rows)
        big = torch.full((T + 2, H), 77, dtype=torch.int8, device="cuda")
        sc = torch.full((T + 2,), -5.0, device="cuda")
        moe.norm_quant_rows(x, "i8", w, r, out=big[:T], scales=sc[:T])
        assert torch.equal(big[:T], out) and (big[T:] == 77).all() and (sc[T:] == -5).all()


# ------------------------------------------------------------------ products

def check_product(y, p, res, dt):
    want = p if res is None else p + res
    bound = 4 * U * np.abs(p) + U * np.abs(want) + store(dt) * np.abs(want) * (1 + 1e-5)
    bad = np.abs(f64(y) - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


SHAPES = [(1, 16, 1), (1, 1536, 4096), (2, 48, 17), (4, 128, 33), (15, 144, 100), (16, 2048, 64),
          (17, 272, 15), (31, 1040, 130), (33, 400, 24), (64, 1536, 48), (65, 1536, 72), (77, 1040, 1001),
          (100, 16, 256), (128, 128, 128), (129, 64, 129), (200, 2064, 384), (255, 80, 257),
          (300, 96, 1000), (513, 1536, 520), (513, 2064, 2041),
          (505, 2064, 1999), (1000, 208, 2000), (1025, 512, 2049), (2500, 4096, 1000),
          (8100, 4112, 2041), (7937, 8192, 2048),
          (16, 1536, 5120), (9, 4112, 8200), (20, 1040, 5001), (32, 4112, 16392), (32, 5136, 1541),
          (5, 4096, 16385), (1, 2064, 32776), (1, 4096, 16384), (64, 5120, 1536), (40, 64, 8199)]


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear_i8(moe, T, K, N):
    for out, with_res in (("bf16", False), ("bf16", True), ("f32", True)):
        print("case: linear", T, K, N, out, with_res, flush=True)
        g = gen(T * 7 + K + N)
        x, sx = codes_of(g, T, K)
        w, sw = codes_of(g, N, K)
        res = torch.randn(T, N, generator=g, device="cuda").to(DT[out]) if with_res else None
        guard = torch.full((T + 1, N), 3.0, dtype=DT[out], device="cuda")
        y = moe.linear_i8(x, sx, w, sw, DT[out], residual=res, y=guard[:T])
        p = f64(x.double() @ w.double().T) * f64(sx)[:, None] * f64(sw)
        check_product(y, p, f64(res) if with_res else None, DT[out])
        assert (guard[T:] == 3).all()
        if with_res:                                     # the residual updated in place
            assert torch.equal(moe.linear_i8(x, sx, w, sw, DT[out], residual=res, y=res), y)


@pytest.mark.parametrize("T,K,N", [(1, 1536, 5120), (4, 48, 33), (16, 2048, 64), (31, 1040, 130),
                                   (64, 272, 48), (100, 1536, 200), (130, 64, 129), (333, 1536, 1040), (333, 1552, 4107),
                                   (1025, 400, 2056), (2500, 2048, 1000),
                                   (8100, 2064, 1021), (7937, 4096, 1024),
                                   (16, 1536, 5119), (3, 1040, 16392), (1, 4112, 8200), (33, 1536, 2560),
                                   (32, 2064, 1030), (9, 144, 4090)])
def test_glu_i8(moe, T, K, N):
    for out in ("bf16", "f32"):
        print("case: glu", T, K, N, out, flush=True)
        g = gen(T + K + N)
        x, sx = codes_of(g, T, K)
        (wg, sg), (wu, su) = codes_of(g, N, K), codes_of(g, N, K)
        sg *= 60.0 / K ** 0.5                # gates to both sides of exp's range
        guard = torch.full((T + 1, N), 3.0, dtype=DT[out], device="cuda")
        h = f64(moe.glu_i8(x, sx, wg, sg, wu, su, DT[out], h=guard[:T]))
        gate = f64(x.double() @ wg.double().T) * f64(sx)[:, None] * f64(sg)
        up = f64(x.double() @ wu.double().T) * f64(sx)[:, None] * f64(su)
        want = gate * mo.sigmoid(gate) * up
        bound = ((12 + 6 * np.abs(gate)) * U + store(DT[out]) * (1 + 1e-4)) * np.abs(want) + 1e-36 * np.abs(up)
        bad = np.abs(h - want) > bound
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
        assert (guard[T:] == 3).all()


def test_linear_extreme_codes(moe):
    """The largest sums: 65536 products of -128 and -128 (2^30), and of -128 and 127."""
    K = 65536
    for T, N in ((1, 5), (40, 20), (200, 140)):
        print("case: extreme", T, N, flush=True)
        x = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
        w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        w[1::2] = 127
        one = torch.ones(max(T, N), device="cuda")
        y = moe.linear_i8(x, one[:T], w, one[:N], torch.float32)
        assert (y[:, 0::2] == 2.0 ** 30).all() and (y[:, 1::2] == -128.0 * 127 * K).all()


def test_linear_rows_do_not_depend_on_the_batch(moe):
    """The sums are exact, so a row has the same bits in any batch."""
    g = gen(5)
    x, sx = codes_of(g, 700, 1552)
    w, sw = codes_of(g, 264, 1552)
    whole = moe.linear_i8(x, sx, w, sw)
    gated = moe.glu_i8(x, sx, w, sw, w, sw)
    for a, b in ((0, 1), (3, 19), (100, 140), (200, 264), (300, 428), (400, 700)):
        print("case: slice", a, b, flush=True)
        assert torch.equal(moe.linear_i8(x[a:b], sx[a:b], w, sw), whole[a:b])
        assert torch.equal(moe.glu_i8(x[a:b], sx[a:b], w, sw, w, sw), gated[a:b])


def test_products_beyond_32_bit_offsets(moe):
    """Row offsets of x (140000 x 16384 codes) and of y (70000 x 32768) past 2^31."""
    g = gen(9)
    T, K, N = 140000, 16384, 24
    x = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(T, generator=g, device="cuda")
    w, sw = codes_of(g, N, K)
    at = torch.tensor([0, 1, 65535, 131071, 131072, 131073, 139998, 139999], device="cuda")
    print("case: long x", flush=True)
    y = moe.linear_i8(x, sx, w, sw, torch.float32)
    p = f64(x[at].double() @ w.double().T) * f64(sx[at])[:, None] * f64(sw)
    check_product(y[at], p, None, torch.float32)
    del x, y
    T, K, N = 70000, 32, 32768
    x, sx = codes_of(g, T, K)
    w, sw = codes_of(g, N, K)
    at = torch.tensor([0, 65535, 65536, 69999], device="cuda")
    print("case: long y", flush=True)
    y = moe.linear_i8(x, sx, w, sw)
    p = f64(x[at].double() @ w.double().T) * f64(sx[at])[:, None] * f64(sw)
    check_product(y[at], p, None, torch.bfloat16)


# ------------------------------------------------------------------ the layer

def layer(g, H, I, act):
    w = {}
    for n, (a, b) in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
        m = torch.randn(a, b, generator=g, device="cuda") * 0.02
        s = m.abs().amax(1) / 127
        w["w_" + n], w["s_" + n] = torch.round(m / s[:, None]).to(torch.int8), s
    return w, (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(DT[act])


def either_side(v, near):
    """int8 codes of v, the same with every code whose quotient is within near(q) of a rounding
    border put on the border's other side, and the scales."""
    c, s = od.quant_i8(v)
    q = v / s[:, None]
    low = np.floor(q)
    return c, np.where(np.abs(q - low - 0.5) <= near(q), 2 * low + 1 - c, c), s


def h16_steps(h):
    """Half a step of int16 codes with one maximum per row and 32 columns, in steps of amax / 127."""
    n = h.shape[1]
    top = np.abs(np.pad(h, ((0, 0), (0, -n % 32)))).reshape(len(h), -1, 32).max(2)
    amax = np.maximum(np.abs(h).max(1, keepdims=True), 1e-300)
    return np.repeat(top, 32, 1)[:, :n] / amax * (127 / 65534)


def layer_and_bound(x, gamma, w, act):
    """The oracle's x_out, its y = x_out - x, and how far from it y may lie, in norm over all rows.

    Everything but the two quantisations is right to some hundred u; a code near a rounding
    border, though, may fall on either side, and that moves its row by a whole step.
      * codes of the normed rows: quotients are off by at most 42 u of themselves (the head of
        this file), so only codes within that of a border differ;
      * h: g and u carry 3 u and the 41 u of their row's scale, so h (12 + 6 |g|) u +
        41 (2 + |g|) u <= (100 + 50 |g|) u; its row's maximum carries as much at its own g, and
        wide batches keep h in 16 bits with half a step of error, h16_steps.
    y' is the oracle with every such code on its border's other side, in both quantisations,
    the second one after the first one's h.  A kernel flips a part of them.  The flips meet
    weights of random signs, so their squares add up: the norm goes as the root of their number.
    A part of the first flips moves h no further than all of them, so the number that it flips
    of h's codes has at most the mean m of y's, a count of rare events: more than 4 times y's
    number and 16 has a chance below 1e-5 at any m (m = 4: 17 or more, 1e-6; m = 8: 17 or more
    where y' has none, 0.004 * 0.0003).  Hence twice |y' - y| and, where a first code can flip,
    the norm of 4 steps of the largest scale at the widest column of w_down in quadrature."""
    def glu(codes, s):
        return od.glu(codes, s, w["w_gate"], w["s_gate"], w["w_up"], w["s_up"])

    c, o, s = either_side(od.norm_rows(x, gamma, None, EPS, act), lambda q: 42 * U * np.abs(q))
    h = glu(c, s)
    g = np.abs(od.product(c, s, w["w_gate"], w["s_gate"]))
    top = np.take_along_axis(g, np.abs(h).argmax(1)[:, None], 1)

    def near(q):
        return (200 + 50 * g + 50 * top) * U * np.abs(q) + h16_steps(h)

    h2 = h if (c == o).all() else glu(o, s)
    y = od.product(*od.quant_i8(h), w["w_down"], w["s_down"])
    _, o2, s2 = either_side(h2, near)
    moved = np.linalg.norm(od.product(o2, s2, w["w_down"], w["s_down"]) - y)
    step = s2.max() * np.linalg.norm(w["w_down"] * w["s_down"][:, None], axis=0).max()
    few = 0 if (c == o).all() else 4 * step
    return x + y, y, np.hypot(2 * moved, few) + 1000 * U * np.linalg.norm(y)


@pytest.mark.parametrize("T,H,I,act", [(1, 1536, 5120, "bf16"), (1, 16, 16, "f32"), (2, 272, 400, "bf16"),
                                       (4, 1536, 4112, "f32"), (9, 2048, 1040, "bf16"), (16, 4096, 8192, "bf16"),
                                       (17, 1536, 512, "bf16"), (16, 4112, 272, "bf16"), (64, 1536, 512, "f32"),
                                       (333, 1536, 4112, "bf16"), (2100, 512, 784, "bf16"), (16, 2048, 32768, "bf16"),
                                       (16, 1536, 5120, "bf16"), (15, 1024, 8192, "f32"), (3, 4096, 32768, "bf16"),
                                       (4090, 2048, 8176, "bf16"), (7900, 2048, 4112, "f32"),
                                       (8, 1536, 8192, "bf16"), (7, 2048, 16384, "f32"), (1, 3488, 4368, "bf16"),
                                       (8, 2048, 80, "f32"), (5, 1488, 112, "bf16"), (1, 2048, 32768, "bf16"),
                                       (8, 2048, 4096, "f32"), (2, 1024, 16384, "bf16"), (3, 512, 8192, "f32")])
def test_dense_layer(moe, T, H, I, act):
    """x_out against the oracle run through all four stages, within layer_and_bound."""
    print("case: layer", T, H, I, act, flush=True)
    dt = DT[act]
    g = gen(T + H + I)
    w, gamma = layer(g, H, I, act)
    x = torch.randn(T, H, generator=g, device="cuda").to(dt)
    cfg = moe.make_dense_config(T, H, I, act)
    ws = moe.alloc_dense_workspace(cfg)
    ws.fill_(0xFF)                                        # the contents on entry are ignored
    wst = moe.dense_weights_struct(w)
    x_in = x.clone()
    got = moe.dense_residual_i8(cfg, x, gamma, wst, ws)
    assert torch.equal(x, x_in)
    ref, y, tol = layer_and_bound(f64(x), f64(gamma), {k: f64(v) for k, v in w.items()}, act)
    err = np.linalg.norm(np.maximum(np.abs(f64(got) - ref) - store(dt) * np.abs(ref) * 1.0001, 0))
    size = np.linalg.norm(y)
    print("rel", err / size, "of", tol / size, flush=True)
    assert err <= tol
    assert tol <= 0.1 * size
    moe.dense_residual_i8(cfg, x, gamma, wst, ws, x_out=x)   # in place, the same bits
    assert torch.equal(x, got)


@pytest.mark.parametrize("T,H,I", [(3, 1536, 1040), (16, 2064, 1040), (90, 512, 784), (700, 1536, 1040),
                                   (4100, 2048, 2064)])
def test_layer_rows_that_are_not_finite(moe, T, H, I):
    """A NaN in one row, an infinity in another: no value of those rows is finite, the others keep
    their bits; then a scale that takes h of every row beyond fp32."""
    print("case: layer, not finite", T, H, I, flush=True)
    g = gen(T + 11)
    w, gamma = layer(g, H, I, "bf16")
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    bad = x.clone()
    bad[0, H - 1], bad[T - 1, 0] = float("nan"), float("-inf")
    cfg = moe.make_dense_config(T, H, I)
    ws, wst = moe.alloc_dense_workspace(cfg), moe.dense_weights_struct(w)
    good, got = (moe.dense_residual_i8(cfg, v, gamma, wst, ws) for v in (x, bad))
    assert torch.equal(good[1:T - 1], got[1:T - 1])
    assert not torch.isfinite(got[0]).any() and not torch.isfinite(got[T - 1]).any()
    w["s_up"][I - 1], w["s_gate"][I - 1] = 1e38, 1.0
    got = moe.dense_residual_i8(cfg, x, gamma, wst, ws)
    acc = f64(moe.linear_i8(*moe.norm_quant_rows(x, "i8", gamma)[:2], w["w_gate"][I - 1:],
                            torch.ones(1, device="cuda"), torch.float32))[:, 0]
    up = f64(moe.linear_i8(*moe.norm_quant_rows(x, "i8", gamma)[:2], w["w_up"][I - 1:],
                           torch.ones(1, device="cuda"), torch.float32))[:, 0]
    over = (acc > 100) & (np.abs(up) > 10)                # silu(g) |u| 1e38 is far beyond fp32
    print("rows beyond fp32:", over.sum(), "of", T, flush=True)
    assert not torch.isfinite(got[torch.from_numpy(over).cuda()]).any()


@pytest.mark.parametrize("T", [64, 700])
def test_layer_is_its_parts(moe, T):
    """norm -> glu -> quantise -> down as four calls, h in fp32.  The codes of the normed rows come
    from the same kernel; a code of h may fall on the other side of a border within the half
    step of h in 16 bits and 8 u of rounding, and as in layer_and_bound the layer is within
    twice of what all of those move."""
    H, I = 1536, 1040
    print("case: parts", T, flush=True)
    g = gen(T)
    w, gamma = layer(g, H, I, "bf16")
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    cfg = moe.make_dense_config(T, H, I)
    whole = moe.dense_residual_i8(cfg, x, gamma, moe.dense_weights_struct(w), moe.alloc_dense_workspace(cfg))
    xq, sx, _ = moe.norm_quant_rows(x, "i8", gamma)
    h = moe.glu_i8(xq, sx, w["w_gate"], w["s_gate"], w["w_up"], w["s_up"], torch.float32)
    hq, sh, _ = moe.norm_quant_rows(h, "i8")
    y = moe.linear_i8(hq, sh, w["w_down"], w["s_down"], torch.float32)
    want = f64(x) + f64(y)
    err = np.maximum(np.abs(f64(whole) - want) - store(torch.bfloat16) * np.abs(want) * 1.0001, 0)
    c, o, s = either_side(f64(h), lambda q: 8 * U * np.abs(q) + h16_steps(f64(h)))
    moved = od.product(o - c, s, f64(w["w_down"]), f64(w["s_down"]))
    err, tol, size = np.linalg.norm(err), 2 * np.linalg.norm(moved), np.linalg.norm(f64(y))
    print("rel", err / size, "of", tol / size, flush=True)
    assert err <= tol + 8 * U * size
    assert tol <= 0.1 * size


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_layer_graph_streams_and_two_workspaces(moe, T):
    """Captured and replayed on changing inputs, and two layers at once on two streams."""
    H, I = 1536, 784
    print("case: graph", T, flush=True)
    g = gen(T + 1)
    w, gamma = layer(g, H, I, "bf16")
    wst = moe.dense_weights_struct(w)
    xs = [torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    cfg = moe.make_dense_config(T, H, I)
    ws = [moe.alloc_dense_workspace(cfg) for _ in range(3)]
    want = [moe.dense_residual_i8(cfg, x, gamma, wst, ws[0]) for x in xs]
    x, y = xs[0].clone(), torch.empty_like(xs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.dense_residual_i8(cfg, x, gamma, wst, ws[0], x_out=y)
    for i in (0, 1, 2, 3, 0, 2):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]), i
        assert torch.equal(moe.dense_residual_i8(cfg, xs[i], gamma, wst, ws[1]), want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[k].append(moe.dense_residual_i8(cfg, xs[1 + k], gamma, wst, ws[1 + k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, want[1 + k]) for o in outs[k])


def test_binding_refuses(moe):
    x, sx = codes_of(gen(1), 4, 64)
    w, sw = codes_of(gen(2), 8, 64)
    for bad in ((x[:, :48], sx, w, sw), (x, sx[:3], w, sw), (x, sx, w.T, sw), (x, sx.half(), w, sw),
                (x.cpu(), sx, w, sw), (x.T.contiguous().T, sx, w, sw)):
        with pytest.raises(ValueError):
            moe.linear_i8(*bad)
    with pytest.raises(moe.MoeError):
        moe.linear_i8(x[:, :40].contiguous(), sx, w[:, :40].contiguous(), sw)   # 40 % 16
    with pytest.raises(ValueError):
        moe.linear_i8(x, sx, w, sw, residual=torch.zeros(4, 8, device="cuda"))  # fp32 for a bf16 y
    with pytest.raises(ValueError):
        moe.glu_i8(x, sx, w, sw, w[:4], sw)
    with pytest.raises(ValueError):
        moe.norm_quant_rows(torch.zeros(4, 64, device="cuda"), "i8", torch.ones(60, device="cuda"))


def test_layer_refuses_weights_of_other_sizes(moe):
    w, gamma = layer(gen(3), 64, 32, "bf16")
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    wst = moe.dense_weights_struct(w)
    for T, I in ((2, 48), (3, 32)):
        cfg = moe.make_dense_config(T, 64, I)
        with pytest.raises(ValueError):
            moe.dense_residual_i8(cfg, x, gamma, wst, moe.alloc_dense_workspace(cfg))
    cfg = moe.make_dense_config(2, 64, 32)
    ws = moe.alloc_dense_workspace(cfg)
    with pytest.raises(moe.MoeError):
        moe.dense_residual_i8(cfg, x, gamma, wst, ws[:256])
    with pytest.raises(ValueError):
        moe.dense_weights_struct(dict(w, w_up=w["w_up"][:16]))
    with pytest.raises(ValueError):
        moe.dense_weights_struct(dict(w, s_down=w["s_gate"]))
    assert torch.equal(moe.dense_residual_i8(cfg, x, gamma, wst, ws), x)      # zero rows stay zero


@pytest.mark.parametrize("T", [4, 300])
def test_dense_layer_then_moe_block(moe, T):
    """The start of a decoder stack: the dense layer 0, then an MoE block on the same residual
    stream, eagerly and as one captured graph; the dense layer against the oracle, the block
    bit for bit against the block run on the dense layer's output by itself."""
    import synth
    from tests.helpers import config_for, to_device
    print("case: stack", T, flush=True)
    shape = synth.WORKLOADS["decode"].with_tokens(T)
    H, I = shape.H, 784
    dev = to_device(synth.make_layer(shape))
    mcfg, mwst = config_for(shape), moe.weights_struct(dev)
    mws = moe.alloc_workspace(mcfg)
    g = gen(T + 5)
    w, gamma = layer(g, H, I, "bf16")
    gamma2 = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    dcfg, dwst = moe.make_dense_config(T, H, I), moe.dense_weights_struct(w)
    dws = moe.alloc_dense_workspace(dcfg)

    def step(x):
        x1 = moe.dense_residual_i8(dcfg, x, gamma, dwst, dws)
        return x1, moe.forward_residual(mcfg, x1, gamma2, None, mws, wst=mwst)

    x = dev["x"].clone()
    x1, x2 = step(x)
    ref, _, tol = layer_and_bound(f64(x), f64(gamma), {k: f64(v) for k, v in w.items()}, "bf16")
    err = np.maximum(np.abs(f64(x1) - ref) - store(torch.bfloat16) * np.abs(ref) * 1.0001, 0)
    assert np.linalg.norm(err) <= tol
    assert torch.equal(moe.forward_residual(mcfg, x1.clone(), gamma2, None, mws, wst=mwst), x2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1, g2 = step(x)
    for _ in range(3):
        g1.zero_()
        g2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g1, x1) and torch.equal(g2, x2)
        step(torch.roll(x, 1, 0).contiguous())                # eager work on the same workspaces
        torch.cuda.synchronize()
