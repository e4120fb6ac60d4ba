"""Packed layers with bias, activation, gate and residual, and their gradient,
on the GPU against the float64 oracle (oracle/layers.py), through the C ABI.

Tolerances, with u = 2^-24 (half a step of fp32, relative) and 2^-8 for bf16:
 * z: the product's bound (product_bound of test_gpu_experts.py, counted there),
   2 u of the magnitudes of a bias, 2^-8 of z where it is kept in bf16.
 * An activation changes by at most 1.13 of what its argument does (the largest
   slope, of gelu). Its own evaluation: the argument of an exponential is off by
   2 u of itself, which the sigmoid's slope turns into at most 2 u 0.23, the
   exponential, the sum and the reciprocal by 2 u each (erfc by 4 u, its argument
   by 2 u); all times |z|: 16 u |z| with room.
 * A gate's product, a residual, a rounding to the type: u, u and 2^-8 (or u).
 * Slopes: at most 1.13, 24 u for their evaluation (sums of two terms of at most
   1.2 and 0.5), times |dY| (and |u|).
 * dX: every dZ is rounded to bf16 once, and so is every weight where dX is bf16,
   2^-8 each of the sum of magnitudes; sums of m products, at most m u of it
   (three products per weight in fp32: (3 m + 3) u).
"""
import numpy as np
import pytest

from oracle import experts as X64
from oracle import layers as L64
from oracle.dequant import dequantize

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import post_weight_quantization_28_amd as G  # noqa: E402
from test_gpu_experts import cuda_layers, expert_ids, layers, product_bound, values  # noqa: E402

U32, UBF = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


def arr(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def last(dtype, x):
    """The last rounding of values of this size."""
    return (UBF if dtype == BF16 else U32) * np.abs(x)


def value_error(name, z, e):
    """Bound on act(z)'s error for a z that is off by e."""
    return (1.13 * e if name != "none" else e) + (0 if name in ("none", "relu") else 16 * U32 * (np.abs(z) + e))


def end_error(name, gated, z, e, residual):
    d = z.shape[1] // 2 if gated else z.shape[1]
    a = L64.act(name, z[:, :d])[0]
    ea = value_error(name, z[:, :d], e[:, :d])
    y, ey = a, ea
    if gated:
        u, eu = z[:, d:], e[:, d:]
        y, ey = a * u, np.abs(u) * ea + np.abs(a) * eu + ea * eu
        ey = ey + U32 * (np.abs(y) + ey)
    if residual is not None:
        ey = ey + U32 * (np.abs(y + residual) + ey)
    return ey


def fast_layers(seed, E, m, n, bits, group):
    qw, sc, zr = layers(seed, E, m, n, bits, group)
    return qw, sc / 4, zr


def linear_bound(X, off, rows, qw, sc, zr, bits, group, n, R, E):
    """product_bound, and up to 48 rows an expert, where either may be taken, the
    larger one of the tiles and of few rows (as counted there)."""
    bound = product_bound(X, off, rows, qw, sc, zr, bits, group, n, R, E)
    if bits == 4 and 16 * E < R <= 48 * E:
        piece = 128 if group % 128 == 0 else 32
        for e in range(len(off) - 1):
            W = np.abs(dequantize(qw[e], sc[e], zr[e], bits, group, n))
            S = np.repeat(np.abs(sc[e].astype(np.float64)), group, axis=1)
            p = slice(off[e], off[e + 1])
            x = np.abs(X[p] if rows is None else X[rows[p]])
            bound[p] = np.maximum(bound[p], U32 * ((piece + 2) * 62 * (x @ S.T) + (n // piece + 1) * (x @ W.T)))
    return bound


LINEARS = [   # T, k, E, d, n, group, drop, only, gathered
    (1, 1, 1, 33, 32, 32, 0.0, None, False),         # one token, one chunk of codes
    (1, 2, 8, 96, 512, 128, 0.0, None, True),
    (3, 1, 1, 128, 1024, 128, 0.0, None, False),     # one dense layer, a few tokens
    (5, 2, 4, 41, 384, 64, 0.0, None, True),         # odd width: rows of Y at any alignment
    (30, 2, 7, 65, 1280, 256, 0.2, None, True),      # dropped slots
    (17, 1, 2, 64, 128, 128, 0.0, [1], True),        # an empty expert
    (20, 2, 8, 50, 1312, 32, 0.1, None, True),       # few rows, small groups
    (40, 2, 4, 100, 96, 96, 0.0, None, True),        # 64-row tiles
    (100, 2, 4, 157, 640, 32, 0.3, None, True),      # ragged both ways
    (600, 1, 2, 3501, 256, 128, 0.1, None, True),    # more tiles
    (300, 2, 2, 7001, 96, 32, 0.0, None, True),      # 128-row tiles
    (257, 2, 3, 96, 320, 160, 0.0, [0, 2], True),    # an empty expert between two
    (30, 4, 2, 70, 2048, 128, 0.1, None, True),      # parts of K
    (90, 1, 1, 33, 4128, 32, 0.0, None, False),
    (17, 1, 1, 70, 2048, 128, 0.0, None, False),     # few rows up to 48 an expert
    (47, 1, 1, 161, 1280, 256, 0.0, None, False),
    (48, 2, 3, 90, 1024, 64, 0.1, None, True),
    (37, 2, 3, 33, 544, 32, 0.1, None, True),
    (70, 1, 3, 4100, 384, 128, 0.0, [0, 1, 2], True),
    (70, 1, 1, 520, 2048, 128, 0.0, None, False),    # tiles with parts of K
    (33, 1, 1, 150, 1088, 64, 0.0, None, False),
    (1200, 1, 2, 6550, 128, 128, 0.1, None, True),   # 256-row tiles (4 bits), ungated 26 of them wide
    (1100, 1, 2, 3201, 384, 128, 0.0, None, False),  # and gated
    (700, 1, 1, 5377, 512, 256, 0.2, None, True),
]


ENDS = [("silu", True), ("gelu", False), ("none", True), ("gelu_tanh", False), ("relu", False), ("none", False)]
# 4 bits with every end, the other widths (whose ends are the same code) and the largest sizes with some
LINEAR_CASES = [c + e + (b,) for c in LINEARS for i, e in enumerate(ENDS) for b in (4, 3, 2)
                if (b == 4 or i < 2) and (c[0] * c[3] < 1000000 or i < 2)]


@pytest.mark.parametrize("T,k,E,d,n,group,drop,only,gathered,name,gated,bits", LINEAR_CASES)
def test_linear(T, k, E, d, n, group, drop, only, gathered, name, gated, bits):
    off, rows, _ = X64.route(expert_ids(T + d, T, k, E, drop, only), E)
    R, m = T * k, 2 * d if gated else d
    X = values(n + T, T if gathered else R, n)
    qw, sc, zr = fast_layers(d + bits, E, m, n, bits, group)
    r = np.random.default_rng(d)
    bias = r.standard_normal((E, m)).astype(np.float32)
    packed = cuda_layers(qw, sc, zr)
    rt = torch.from_numpy(rows).cuda() if gathered else None
    seg = None if E == 1 and drop == 0 else torch.from_numpy(off).cuda()
    src = rows if gathered else None
    bound = linear_bound(arr(X), off, src, qw, sc, zr, bits, group, n, R, E)
    live = slice(0, off[-1])
    for i, (ydt, rdt, zdt) in enumerate([(BF16, BF16, BF16), (F32, F32, F32), (BF16, None, None), (F32, BF16, None)]):
        if bits != 4 and i > 1:
            break
        res = None if rdt is None else values(5, R, d, dtype=rdt)
        b = None if i == 2 else bias
        out, kept = values(8, R, d, dtype=ydt), None if zdt is None else values(9, R, m, dtype=zdt)
        before, zbefore = arr(out), np.zeros((R, m)) if kept is None else arr(kept)
        got = G.linear(X, *packed, bits, group, bias=None if b is None else torch.from_numpy(b).cuda(), act=name,
                       gated=gated, residual=res, offsets=seg, rows=rt, keep=kept, out=out)
        Y, Z = got if kept is not None else (got, None)
        assert Y is out and (kept is None or Z is kept)
        ref, zref = L64.linear(arr(X), off, qw, sc, zr, bits, group, name, gated, before, zbefore, b,
                               None if res is None else arr(res), src)
        e = bound + (0 if b is None else 2 * U32 * (np.abs(zref) + np.abs(np.repeat(bias, np.diff(off), axis=0)).max()))
        ey = end_error(name, gated, zref, e, None if res is None else arr(res))
        ey = ey + last(ydt, np.abs(ref) + ey)
        assert np.all((np.abs(arr(Y) - ref) <= ey)[live])
        assert np.array_equal(arr(Y)[off[-1]:], before[off[-1]:])
        if kept is not None:
            assert np.all((np.abs(arr(Z) - zref) <= e + last(zdt, np.abs(zref) + e))[live])
            assert np.array_equal(arr(Z)[off[-1]:], zbefore[off[-1]:])


# A wave of the matrix-vector form holds the scales of 8 groups at a time: sizes at
# which it comes back for more, in four loads of one and one of four.
MANY_GROUPS = [   # T, k, E, d, n, group, drop, only, gathered
    (3, 1, 1, 70, 10880, 128, 0.0, None, False),     # eight waves, 11 groups each; 85 groups of a row
    (12, 1, 1, 33, 9728, 128, 0.0, None, False),     # 76 groups, 10 each
    (5, 2, 4, 40, 18688, 256, 0.0, None, True),      # eight waves, 10 groups of 256 each
    (40, 1, 1, 40, 10880, 128, 0.0, None, False),    # three tiles of 16 rows
]


@pytest.mark.parametrize("bits", [4, 3, 2])
@pytest.mark.parametrize("case", MANY_GROUPS, ids=str)
def test_linear_of_many_groups_a_wave(case, bits):
    for name, gated in ENDS[:2]:
        test_linear(*case, name, gated, bits)


def test_linear_of_many_groups_in_many_workgroups():
    """More than 512 of them: four waves, 10 groups each."""
    test_linear(500, 1, 32, 135, 4736, 128, 0.0, None, True, "silu", True, 4)


GRADS = [   # R, E, d, n, group, cuts (None: one layer without offsets)
    (1, 1, 32, 64, 32, None), (1, 1, 1, 32, 32, None), (3, 2, 70, 128, 128, [1, 3]), (50, 3, 65, 96, 96, [20, 20, 45]),
    (130, 1, 64, 160, 32, None), (400, 2, 257, 320, 64, [129, 400]), (300, 2, 100, 256, 256, [0, 290]),
    (1100, 2, 96, 320, 64, [500, 1090]), (24, 4, 750, 128, 32, [3, 3, 10, 23]), (20, 1, 1501, 96, 32, None),
    (700, 70, 40, 64, 32, "many"), (64, 1, 300, 64, 32, [64]), (65, 1, 256, 64, 64, [65]), (1100, 2, 96, 6432, 32, [500, 1090]),
]


def segments(E, R, cuts):
    if cuts == "many":                                       # more than 64 segments, some empty
        return np.r_[0, np.sort(np.random.default_rng(E).integers(0, R - 5, E))].astype(np.int32)
    return np.array([0] + (cuts if cuts is not None else [R]), np.int32)


GRAD_ENDS = [("silu", True), ("gelu", False), ("gelu_tanh", True), ("relu", False), ("none", False), ("none", True)]
GRAD_CASES = [c + e + (b,) for c in GRADS for i, e in enumerate(GRAD_ENDS) for b in (4, 3) if b == 4 or i == 0]


@pytest.mark.parametrize("R,E,d,n,group,cuts,name,gated,bits", GRAD_CASES)
def test_linear_grad(R, E, d, n, group, cuts, name, gated, bits):
    off = segments(E, R, cuts)
    m = 2 * d if gated else d
    qw, sc, zr = layers(d + bits, E, m, n, bits, group)
    packed = cuda_layers(qw, sc, zr)
    live = slice(off[0], off[-1])
    per = np.diff(off).max() if E else 0
    for dydt, zdt, xdt in ((BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16), (F32, BF16, BF16)):
        dY, Z = values(1, R, d, dtype=dydt, scale=1e-2), values(2, R, m, dtype=zdt, scale=1.5)
        dZ, out = values(3, R, m), values(4, R, n, dtype=xdt)
        zb, xb = arr(dZ), arr(out)
        dX, dZ2, db = G.linear_grad(dY, Z, *packed, bits, group, n, act=name, gated=gated,
                                    offsets=None if cuts is None else torch.from_numpy(off).cuda(), want_bias=True, dZ=dZ,
                                    out=out)
        assert dX is out and dZ2 is dZ
        rx, rz, rb = L64.linear_grad(arr(dY), arr(Z), off, qw, sc, zr, bits, group, n, name, gated, zb, xb)
        g, z = np.abs(arr(dY)), np.abs(arr(Z))
        if gated:
            f = np.concatenate([g * z[:, d:], g * z[:, :d]], axis=1)   # what slope or value are multiplied by, or bound by
        else:
            f = g
        ez = (0 if name == "none" and not gated else 32 * U32) * f
        assert np.all((np.abs(arr(dZ) - rz) <= ez + UBF * (np.abs(rz) + ez) + 2.0 ** -134)[live])
        assert np.array_equal(arr(dZ)[off[-1]:], zb[off[-1]:])
        eb = np.zeros_like(rb)
        for e in range(E):
            p = slice(off[e], off[e + 1])
            # at most per / 8 + 8 + per / 64 additions in one chain
            eb[e] = ez[p].sum(0) if not np.isscalar(ez) else 0
            eb[e] += U32 * (per / 8 + per / 64 + 12) * np.abs(rz[p]).sum(0)
        assert np.all(np.abs(arr(db) - rb) <= eb)
        mag = np.zeros((R, n))
        ezx = np.zeros((R, n))
        for e in range(E):
            p, W = slice(off[e], off[e + 1]), np.abs(dequantize(qw[e], sc[e], zr[e], bits, group, n))
            mag[p] = np.abs(rz[p]) @ W
            ezx[p] = (ez[p] if not np.isscalar(ez) else np.zeros_like(rz[p])) @ W
        ex = 1.01 * (ezx + UBF * mag) + ((UBF + (m + 2) * U32) if xdt == BF16 else (3 * m + 3) * U32) * 1.01 * mag
        assert np.all((np.abs(arr(dX) - rx) <= ex + last(xdt, np.abs(rx) + ex))[live])
        assert np.array_equal(arr(dX)[off[-1]:], xb[off[-1]:])


def test_gelu_in_its_tail():
    """Below z = -2, where Phi is a small difference of the slope's terms: value
    and slope keep their relative precision. With x = z^2 / 2 the exponential's
    argument is off by at most 3 u of itself, the other factors by 20 u together;
    Phi is at most a quarter of |z| phi, so their difference is off by at most
    (1 + 1/4) / (1 - 1/4) < 2 times as much, relative to itself."""
    from scipy.special import erfc
    z = np.linspace(-12, -2, 4096).astype(np.float32).astype(np.float64)
    qw, sc, zr = layers(1, 1, 8192, 32, 4, 32)
    packed = cuda_layers(qw, sc, zr)
    phi, cdf = np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi), 0.5 * erfc(-z / np.sqrt(2))
    rel = UBF + 1.01 * (3 * 0.5 * z * z + 20) * U32
    Z = torch.from_numpy(np.stack([np.concatenate([z, np.ones_like(z)])])).float().cuda()
    dY = torch.ones((1, 4096), device="cuda")
    _, dZ, _ = G.linear_grad(dY, Z, *packed, 4, 32, 32, act="gelu", gated=True)
    got = arr(dZ)[0]
    slope = cdf + z * phi
    assert np.all(np.abs(got[:4096] - slope) <= 2 * rel * np.abs(slope))
    assert np.all(np.abs(got[4096:] - z * cdf) <= rel * np.abs(z * cdf))


def test_silu_in_its_tail():
    """z from the bias alone, in fp32: relative to itself silu is off by 1.3 |z| u for
    z < 0 (the rounding of z log2 e, and of log2 e itself, in the exponent), and by the
    exponential's, the sum's, the reciprocal's, the product's and the result's 10 u."""
    z = np.linspace(-80, 20, 8192).astype(np.float32)
    packed = cuda_layers(*layers(1, 1, 8192, 32, 4, 32))
    X = torch.zeros((1, 32), dtype=BF16, device="cuda")
    Y = arr(G.linear(X, *packed, 4, 32, bias=torch.from_numpy(z[None]).cuda(), act="silu", out_dtype=F32))[0]
    z64 = z.astype(np.float64)
    ref = z64 / (1 + np.exp(-z64))
    assert np.all(np.abs(Y - ref) <= U32 * (1.3 * np.maximum(-z64, 0) + 10) * np.abs(ref))


def test_linear_grad_of_a_plain_layer_needs_no_copy():
    """No activation, no gate: dY stands for dZ, Z is not read; an fp32 dY is
    rounded into a new dZ; an expert without rows has a bias gradient of zero."""
    qw, sc, zr = layers(1, 3, 70, 128, 4, 64)
    packed = cuda_layers(qw, sc, zr)
    off = torch.tensor([0, 40, 40, 90], dtype=torch.int32, device="cuda")
    dY = values(1, 90, 70)
    dX, dZ, db = G.linear_grad(dY, None, *packed, 4, 64, 128, offsets=off, want_bias=True)
    assert dZ is dY and torch.equal(dX, G.expert_matmul_grad(dY, off, *packed, 4, 64, 128))
    assert torch.count_nonzero(db[1]) == 0 and db.shape == (3, 70)
    a, b, c = G.linear_grad(dY.float(), None, *packed, 4, 64, 128, offsets=off)
    assert torch.equal(b, dY) and torch.equal(a, dX) and c is None
    x, z, db = G.linear_grad(dY[:0], None, *packed, 4, 64, 128, offsets=off * 0, want_bias=True)
    assert x.shape == (0, 128) and torch.count_nonzero(db) == 0


def test_residual_and_gradients_in_place():
    """Y over the residual, dZ over Z and over dY."""
    qw, sc, zr = fast_layers(1, 1, 128, 256, 4, 64)
    packed = cuda_layers(qw, sc, zr)
    for R in (3, 40, 300):
        X, res = values(R, R, 256), values(2, R, 64)
        want = G.linear(X, *packed, 4, 64, act="silu", gated=True, residual=res)
        got = G.linear(X, *packed, 4, 64, act="silu", gated=True, residual=res, out=res)
        assert got is res and torch.equal(res, want)
        dY, Z = values(3, R, 64), values(4, R, 128)
        want = G.linear_grad(dY, Z, *packed, 4, 64, 256, act="silu", gated=True)
        got = G.linear_grad(dY, Z, *packed, 4, 64, 256, act="silu", gated=True, dZ=Z)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], Z)
        dY, Z = values(3, R, 128), values(4, R, 128)
        want = G.linear_grad(dY, Z, *packed, 4, 64, 256, act="gelu", want_bias=True)
        got = G.linear_grad(dY, Z, *packed, 4, 64, 256, act="gelu", dZ=dY, want_bias=True)
        assert torch.equal(want[1], dY) and torch.equal(want[0], got[0]) and torch.equal(want[2], got[2])


def test_linear_at_any_alignment():
    """Rows apart and at odd addresses: the aligned result within the last
    rounding's and the sums' bounds, nothing written beside the rows."""
    n, d, E = 256, 33, 1
    for R in (5, 50, 300):
        for gated in (False, True):
            m = 2 * d if gated else d
            qw, sc, zr = fast_layers(R, E, m, n, 4, 128)
            packed = cuda_layers(qw, sc, zr)
            X, res = values(R, R, n), values(3, R, d)
            wx, wr = values(4, R, n + 5), values(5, R, d + 3)
            wx[:, 3:3 + n], wr[:, 1:1 + d] = X, res
            wy = torch.full((R, d + 9), 7.0, dtype=BF16, device="cuda")
            wz = torch.full((R, m + 4), 7.0, dtype=F32, device="cuda")
            Y, Z = G.linear(X, *packed, 4, 128, act="gelu", gated=gated, residual=res, keep=F32)
            G.linear(wx[:, 3:3 + n], *packed, 4, 128, act="gelu", gated=gated, residual=wr[:, 1:1 + d],
                     keep=wz[:, 2:2 + m], out=wy[:, 4:4 + d])
            # (unaligned rows go in tiles, whose bound is the smaller one)
            e = 2 * product_bound(arr(X), [0, R], None, qw, sc, zr, 4, 128, n, R, 1)
            assert np.all(np.abs(arr(wz[:, 2:2 + m]) - arr(Z)) <= e)
            ey = 2 * end_error("gelu", gated, arr(Z), e, arr(res))
            assert np.all(np.abs(arr(wy[:, 4:4 + d]) - arr(Y)) <= ey + 2 * last(BF16, np.abs(arr(Y)) + ey))
            assert torch.all(wy[:, :4] == 7) and torch.all(wy[:, 4 + d:] == 7)
            assert torch.all(wz[:, :2] == 7) and torch.all(wz[:, 2 + m:] == 7)


def test_more_packed_rows_than_the_matrix_vector_form_has_threads_for():
    """17 rows at 3 bits go by that form, eight threads a packed row, while they
    are below 2^32: 2^29 + 64 packed rows go in tiles."""
    m, n, R = 2 ** 29 + 64, 32, 17
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    qw = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, m, 3), generator=g, device="cuda", dtype=torch.int32)
    sc = torch.rand((1, m, 1), generator=g, device="cuda") + 0.5
    zr = torch.randint(0, 8, (1, m, 1), generator=g, device="cuda", dtype=torch.uint8)
    X = values(1, R, n)
    Y = G.linear(X, qw, sc, zr, 3, 32)
    for at in (slice(0, 200), slice(2 ** 28 - 100, 2 ** 28 + 100), slice(m - 200, m)):
        w = [t[:, at].cpu().numpy() for t in (qw, sc, zr)]
        w[0] = w[0].view(np.uint32)
        ref = arr(X) @ dequantize(w[0][0], w[1][0], w[2][0], 3, 32, n).T
        e = product_bound(arr(X), [0, R], None, *w, 3, 32, n, R, 1)
        assert np.all(np.abs(arr(Y[:, at]) - ref) <= e + last(BF16, np.abs(ref) + e))


def test_nonfinite_activations_stay_in_their_rows():
    for R in (6, 60, 400):
        X = values(R, R, 128)
        X[2, 5], X[4, 7] = float("nan"), float("inf")
        qw, sc, zr = fast_layers(1, 1, 96, 128, 4, 32)
        for name in L64_ACTS:
            Y = arr(G.linear(X, *cuda_layers(qw, sc, zr), 4, 32, act=name))
            bad = ~np.isfinite(Y).all(1)
            assert np.isnan(Y[2]).all() and set(np.nonzero(bad)[0]) <= {2, 4}
            assert bad[4] or name == "relu"


L64_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def test_activations_over_their_range():
    """Values and slopes from large negative to large positive arguments, through
    a layer that is the identity (code 1, zero point 0, scale 1)."""
    n = 32
    codes = np.eye(n, dtype=np.uint8)
    from oracle import packing as P
    packed = cuda_layers(P.pack(codes, 4)[None], np.ones((1, n, 1), np.float32), np.zeros((1, n, 1), np.uint8))
    z = np.concatenate([np.linspace(-12, 12, 2001), [-3e4, -200.0, -90.0, 0.0, 90.0, 200.0, 3e4], -2.0 ** np.arange(-40, 5.0)])
    z = np.resize(z, (-(-len(z) // n)) * n).reshape(-1, n)
    X = torch.from_numpy(z.astype(np.float32)).to(BF16).cuda()
    zz = arr(X)
    for name in L64_ACTS:
        Y, Z = G.linear(X, *packed, 4, 32, act=name, keep=F32, out_dtype=F32)
        assert np.array_equal(arr(Z), zz)
        with np.errstate(over="ignore"):
            a, slope = L64.act(name, zz)
        assert np.all(np.abs(arr(Y) - a) <= 16 * U32 * np.abs(zz))
        dY = torch.ones_like(Z)
        _, dZ, db = G.linear_grad(dY, Z, *packed, 4, 32, n, act=name, want_bias=True)
        assert np.all(np.abs(arr(dZ) - slope) <= 32 * U32 + UBF * np.abs(slope) + 2.0 ** -134)
        assert np.all(np.abs(arr(db)[0] - slope.sum(0)) <= (32 + 40) * U32 * (1.2 * len(zz)))


def test_gradients_against_differences():
    """Adjoint: <dY, linear(X + h V) - linear(X - h V)> / 2 h = <dX, V> in the
    oracle's forward, for a gated layer of two experts."""
    R, E, d, n, group = 30, 2, 32, 64, 32
    off = np.array([0, 13, 30], np.int32)
    qw, sc, zr = fast_layers(3, E, 2 * d, n, 4, group)
    packed = cuda_layers(qw, sc, zr)
    X = values(1, R, n)
    seg = torch.from_numpy(off).cuda()
    _, Z = G.linear(X, *packed, 4, group, act="silu", gated=True, offsets=seg, keep=F32)
    dY = values(2, R, d)
    dX, _, db = G.linear_grad(dY, Z, *packed, 4, group, n, act="silu", gated=True, offsets=seg, want_bias=True,
                              out_dtype=F32)
    r = np.random.default_rng(5)
    V = r.standard_normal((R, n))

    def total(x, bias):
        return float((L64.linear(x, off, qw, sc, zr, 4, group, "silu", True, np.zeros((R, d)), np.zeros((R, 2 * d)),
                                 bias)[0] * arr(dY)).sum())
    h = 1e-4
    zero = np.zeros((E, 2 * d))
    diff = (total(arr(X) + h * V, zero) - total(arr(X) - h * V, zero)) / (2 * h)
    z = arr(Z)
    W = [np.abs(dequantize(qw[e], sc[e], zr[e], 4, group, n)) for e in range(E)]
    dz = np.abs(L64.linear_grad(arr(dY), z, off, qw, sc, zr, 4, group, n, "silu", True, np.zeros_like(z), np.zeros((R, n)))[1])
    mag = sum((dz[off[e]:off[e + 1]] @ W[e] * np.abs(V[off[e]:off[e + 1]])).sum() for e in range(E))
    # dZ rounded to bf16: 2^-8 of the magnitudes; the difference itself: h^2 of third derivatives, far below
    assert abs(float((arr(dX) * V).sum()) - diff) <= (UBF + 1e-4) * mag
    B = r.standard_normal((E, 2 * d))
    diff = (total(arr(X), h * B) - total(arr(X), -h * B)) / (2 * h)
    big = sum((dz[off[e]:off[e + 1]] * np.abs(B[e])).sum() for e in range(E))
    assert abs(float((arr(db) * B).sum()) - diff) <= 1e-4 * big


def test_wrong_offsets_stay_in_bounds():
    """Offsets that fall, pass R or are negative give some result and touch
    nothing outside the matrices."""
    qw, sc, zr = fast_layers(1, 4, 64, 64, 4, 32)
    packed = cuda_layers(qw, sc, zr)
    for bad in ([0, 30, 10, 90, 40], [-5, 3, 3, 1000, 2000], [50, 40, 30, 20, 10]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        rows = torch.tensor([-7, 10 ** 9] * 25, dtype=torch.int32, device="cuda")
        bias = torch.ones(4, 64, device="cuda")
        pad = torch.full((60, 40), 3.0, dtype=BF16, device="cuda")
        out, kept = pad[5:55, :32], torch.full((60, 70), 3.0, dtype=BF16, device="cuda")
        G.linear(values(1, 9, 64), *packed, 4, 32, bias=bias, act="silu", gated=True, offsets=off, rows=rows, out=out,
                 keep=kept[5:55, :64])
        dz = torch.full((60, 70), 3.0, dtype=BF16, device="cuda")
        G.linear_grad(values(2, 50, 32), values(3, 50, 64), *packed, 4, 32, 64, act="silu", gated=True, offsets=off,
                      want_bias=True, dZ=dz[5:55, :64])
        torch.cuda.synchronize()
        for t, w in ((pad, 32), (kept, 64), (dz, 64)):
            assert torch.all(t[:5] == 3) and torch.all(t[55:] == 3) and torch.all(t[:, w:] == 3)


@pytest.mark.parametrize("E,R,off", [
    (4, 3200, [0, 3200, 0, 3200, 0]),                        # two segments of all rows: 200 tiles of 32 rows, sums for 103
    (4, 50, [0, 50, 0, 50, 0]), (3, 3, [0, 3, 0, 3]),
    (130, 2000, [0, 2000] * 65 + [0]), (70, 96, [96, 0] * 35 + [96]),
])
def test_overlapping_segments_have_no_sums_beyond_their_tiles(E, R, off):
    """Offsets that fall make segments overlap, with more tiles of 32 rows between
    them than there are sums for (min(R, R / 32 + E - 1)): those that there are count,
    in order, and nothing is read behind them (the bytes there are NaN)."""
    n, m, tiles = 32, 33, min(R, -(-R // 32) + E - 1)
    packed = cuda_layers(*layers(1, E, m, n, 4, 32))
    dY = values(1, R, m)
    need = G.gptq._bytes("gptq_linear_grad_workspace_bytes", R, n, m, 0, E, 4, 32)
    first, want, mag = 0, np.zeros((E, m)), np.zeros((E, m))
    for e in range(E):
        lo = min(max(off[e], 0), R)
        hi = min(max(off[e + 1], lo), R)
        count = min(-(-(hi - lo) // 32), tiles - first)
        p = slice(lo, min(hi, lo + 32 * count))
        want[e], mag[e] = arr(dY)[p].sum(0), np.abs(arr(dY)[p]).sum(0)
        first += count
        assert 0 <= count and first <= tiles and 4 * first * m <= need
    ws = torch.full((need + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    _, _, db = G.linear_grad(dY, None, *packed, 4, 32, n, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"),
                             want_bias=True, workspace=ws[:need])
    assert np.all(np.abs(arr(db) - want) <= U32 * (R / 8 + R / 64 + 12) * mag)
    assert torch.all(ws[need:] == 255)


@pytest.mark.parametrize("T", [4, 600])
def test_captured_step_replays(T):
    """Forward and backward in a captured graph, replayed on changing inputs
    with eager work between: bitwise the eager results."""
    E, d, n, group = 4, 96, 256, 128
    qw, sc, zr = fast_layers(1, E, 2 * d, n, 4, group)
    packed = cuda_layers(qw, sc, zr)
    off, rows, _ = X64.route(expert_ids(T, T, 2, E), E)
    seg, src = torch.from_numpy(off).cuda(), torch.from_numpy(rows).cuda()
    res, dY = values(4, 2 * T, d), values(5, 2 * T, d)

    def step(x):
        Y, Z = G.linear(x, *packed, 4, group, act="silu", gated=True, residual=res, offsets=seg, rows=src, keep=BF16)
        return (Y, Z) + G.linear_grad(dY, Z, *packed, 4, group, n, act="silu", gated=True, offsets=seg, want_bias=True)
    X = [values(10 + i, T, n) for i in range(3)]
    want = [[t.clone() for t in step(x)] for x in X]
    live = X[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(live)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(live)
    for i in (0, 1, 2, 0):
        live.copy_(X[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        step(X[1])


def test_two_streams_at_once():
    """The same layers on two streams, whose calls have their own workspaces."""
    E, n, d = 4, 256, 128
    up, down = fast_layers(1, E, 2 * d, n, 4, 64), fast_layers(2, E, n, d, 4, 64)
    pu, pd = cuda_layers(*up), cuda_layers(*down)
    dense = cuda_layers(*fast_layers(3, 1, 70, 2048, 4, 64))
    ids = torch.from_numpy(expert_ids(4, 6, 2, E, 0.1, None)).cuda()
    inputs = [(values(10 + i, 6, n), values(20 + i, 70, 2048), values(30 + i, 70, 70), values(40 + i, 70, 70)) for i in range(2)]

    def step(x, wide, dy, z):
        return (G.expert_layer(x, ids, None, pu, pd, 4, 64), G.linear(wide, *dense, 4, 64, act="silu"),
                *G.linear_grad(dy, z, *dense, 4, 64, 2048, act="silu", want_bias=True))

    want = [step(*i) for i in inputs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(*inputs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_a_tuning_step_end_to_end():
    """An MLP of packed layers under a distillation loss, as a tuning step runs it:
    linear (gated, z kept), linear (bias, residual), a packed head, distill, and
    back. Every output against the oracle on the same inputs as the call had, and
    the loss' change along the final gradient against the gradient's own length."""
    T, n, d, V, K, group = 50, 128, 96, 352, 7, 32
    up, down, head = fast_layers(1, 1, 2 * d, n, 4, group), fast_layers(2, 1, n, d, 4, group), fast_layers(3, 1, V, n, 4, group)
    pu, pd, ph = cuda_layers(*up), cuda_layers(*down), cuda_layers(*head)
    off = [0, T]
    r = np.random.default_rng(9)
    X = values(1, T, n, scale=0.3)
    bias = torch.from_numpy(r.standard_normal((1, n)).astype(np.float32)).cuda()
    ids = torch.from_numpy(np.stack([r.choice(V, K, replace=False) for _ in range(T)]).astype(np.int32)).cuda()
    teacher = torch.from_numpy((2 * r.standard_normal((T, K))).astype(np.float32)).cuda()
    g = torch.full((T,), 1.0 / T, device="cuda")
    h, z = G.linear(X, *pu, 4, group, act="silu", gated=True, keep=BF16)
    y = G.linear(h, *pd, 4, group, bias=bias, residual=X)
    logits = G.linear(y, *ph, 4, group, out_dtype=F32)
    loss, lse = G.distill(logits, ids, teacher)
    dl = G.distill_grad(logits, ids, teacher, lse, g, out_dtype=BF16)
    dy, _, _ = G.linear_grad(dl, None, *ph, 4, group, n)
    dh, _, db = G.linear_grad(dy, None, *pd, 4, group, d, want_bias=True)
    dx, dz, _ = G.linear_grad(dh, z, *pu, 4, group, n, act="silu", gated=True)

    def forward(x):
        hh, zz = L64.linear(x, off, *up, 4, group, "silu", True, np.zeros((T, d)), np.zeros((T, 2 * d)))
        yy, _ = L64.linear(hh, off, *down, 4, group, "none", False, np.zeros((T, n)), np.zeros((T, n)), arr(bias), x)
        ll, _ = L64.linear(yy, off, *head, 4, group, "none", False, np.zeros((T, V)), np.zeros((T, V)))
        return hh, zz, yy, ll, L64.distill(ll, ids.cpu().numpy(), arr(teacher), 1.0, False)
    x64 = arr(X)
    hh, zz, yy, ll, (l64, e64, ps) = forward(x64)
    # what rounding h, z and y to bf16 may do downstream: 2^-8 of the magnitudes that the weights add up
    Wd, Wh = np.abs(dequantize(down[0][0], down[1][0], down[2][0], 4, group, d)), np.abs(dequantize(head[0][0], head[1][0], head[2][0], 4, group, n))
    eh = 1.01 * UBF * np.abs(hh) + 1e-5 * (1 + np.abs(hh))
    assert np.all(np.abs(arr(h) - hh) <= eh) and np.all(np.abs(arr(z) - zz) <= 1.01 * UBF * np.abs(zz) + 1e-5)
    ey = 1.01 * (eh @ Wd.T) + 1.01 * UBF * np.abs(yy) + 1e-5 * (1 + np.abs(yy))
    assert np.all(np.abs(arr(y) - yy) <= ey)
    el = 1.01 * (ey @ Wh.T) + 1e-4
    assert np.all(np.abs(arr(logits) - ll) <= el)
    # a loss and its lse change by at most twice and once the largest change of a row's logits
    assert np.all(np.abs(arr(lse) - e64) <= el.max(1) + 1e-5) and np.all(np.abs(arr(loss) - l64) <= 2 * el.max(1) + 1e-5)
    # the way back, each call on what it was given
    got_l = arr(logits)
    _, e2, p2 = L64.distill(got_l, ids.cpu().numpy(), arr(teacher), 1.0, False)
    ref = L64.distill_grad(got_l, e2, p2, arr(g), 1.0)
    assert np.all(np.abs(arr(dl) - ref) <= 1.01 * UBF * np.abs(ref) + 1e-5 / T)
    for got, grad, zin, packed, width, name, gated in ((dy, dl, None, head, n, "none", False), (dh, dy, None, down, d, "none", False),
                                                       (dx, dh, z, up, n, "silu", True)):
        m = packed[0].shape[1]
        rx, rz, rb = L64.linear_grad(arr(grad), None if zin is None else arr(zin), off, *packed, 4, group, width, name, gated,
                                     np.zeros((T, m)), np.zeros((T, width)))
        W = np.abs(dequantize(packed[0][0], packed[1][0], packed[2][0], 4, group, width))
        assert np.all(np.abs(arr(got) - rx) <= (2 * UBF + 1e-4) * (np.abs(rz) @ W) + UBF * np.abs(rx) + 1e-12)
    assert np.all(np.abs(arr(db)[0] - arr(dy).sum(0)) <= (T + 4) * U32 * np.abs(arr(dy)).sum(0))
    # along the gradient (with the residual's share) the oracle's loss changes by its squared length
    full = arr(dx) + arr(dy)
    step = 1e-3 / np.abs(full).max()
    diff = (forward(x64 + step * full)[4][0].mean() - forward(x64 - step * full)[4][0].mean()) / (2 * step)
    length = float((full * full).sum())
    # the chain's roundings: six at most, 2^-8 each of magnitudes that add up to several times the gradient's own
    assert abs(diff - length) <= 0.05 * length


def test_linear_binding_refusals():
    qw, sc, zr = cuda_layers(*fast_layers(1, 2, 64, 64, 4, 32))
    X, off = values(1, 6, 64), torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    ok = dict(act="silu", gated=True, offsets=off)
    G.linear(X, qw, sc, zr, 4, 32, **ok)
    for bad in (dict(act="tanh"), dict(act=None), dict(bias=torch.zeros(2, 32, device="cuda")), dict(residual=values(1, 6, 64)),
                dict(keep=values(1, 6, 32)), dict(out=values(1, 6, 64)), dict(offsets=off[:2])):
        with pytest.raises(ValueError):
            G.linear(X, qw, sc, zr, 4, 32, **{**ok, **bad})
    for bad in (dict(bias=torch.zeros(2, 64, dtype=BF16, device="cuda")), dict(residual=values(1, 6, 32).half()),
                dict(keep=torch.float16), dict(out_dtype=torch.float16), dict(bias=torch.zeros(2, 64))):
        with pytest.raises(TypeError):
            G.linear(X, qw, sc, zr, 4, 32, **{**ok, **bad})
    odd = cuda_layers(*fast_layers(1, 1, 33, 64, 4, 32))
    with pytest.raises(ValueError):
        G.linear(X, *odd, 4, 32, act="silu", gated=True)
    dY = values(1, 6, 32)
    with pytest.raises(ValueError):
        G.linear_grad(dY, None, qw, sc, zr, 4, 32, 64, **ok)
    with pytest.raises(ValueError):
        G.linear_grad(values(1, 6, 64), values(1, 6, 64), qw, sc, zr, 4, 32, 64, **ok)
    with pytest.raises(ValueError):
        G.linear_grad(dY, values(1, 6, 32), qw, sc, zr, 4, 32, 64, **ok)
    with pytest.raises(TypeError):
        G.linear_grad(dY, values(1, 6, 64), qw, sc, zr, 4, 32, 64, dZ=torch.zeros(6, 64, device="cuda"), **ok)


# ---------------------------------------------------------------- a layer of experts for a few tokens
def layer_bound(X, ids, w, up, down, bits, group, name, gated, b1, b2, res, pieces):
    """Bound on expert_layer's fp32 sum, slot by slot: z and the product with h as
    the matrix-vector form of product_bound, the activation's as above, h rounded to
    bf16 (2^-8) or held in three pieces (u), k fused sums, a bias, the residual."""
    T, k = ids.shape
    E, n, d = up[0].shape[0], X.shape[1], up[0].shape[1] // (2 if gated else 1)
    out = np.zeros((T, n))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            one = [0, 1]
            x = np.abs(X[t:t + 1])
            ez = product_bound(x, one, None, *(a[e:e + 1] for a in up), bits, group, n, 1, 1)
            z = X[t:t + 1] @ dequantize(up[0][e], up[1][e], up[2][e], bits, group, n).T
            if b1 is not None:
                z = z + b1[e]
                ez = ez + 2 * U32 * (np.abs(z) + np.abs(b1[e]))
            eh = end_error(name, gated, z, ez, None)
            h = L64.end(z, name, gated)
            eh = eh + (UBF if pieces == 1 else 2 * U32) * (np.abs(h) + eh)
            D = np.abs(dequantize(down[0][e], down[1][e], down[2][e], bits, group, d))
            # the parts of K and the three pieces add at most as many sums again
            eo = eh @ D.T + 3 * product_bound(np.abs(h) + eh, one, None, *(a[e:e + 1] for a in down), bits, group, d, 1, 1)
            o = np.abs(h) @ D.T + (0 if b2 is None else np.abs(b2[e]))
            out[t] += abs(float(w[t, j])) * (eo + (k + 3) * U32 * (o + eo))[0]
        if res is not None:
            out[t] += U32 * np.abs(res[t])
    return out


LAYERS = [   # T, k, E, n, d, group, drop, bias
    (1, 1, 1, 32, 32, 32, 0.0, True), (1, 2, 8, 256, 384, 128, 0.0, False), (1, 8, 64, 128, 256, 128, 0.0, True),
    (1, 3, 2, 96, 160, 32, 0.0, False),              # an expert twice in a row
    (2, 2, 4, 640, 128, 64, 0.0, True), (5, 2, 3, 128, 96, 32, 0.3, True), (17, 1, 1, 256, 128, 128, 0.0, False),
    (40, 2, 3, 128, 384, 128, 0.1, True),            # more than one tile an expert
    (16, 4, 100, 64, 64, 64, 0.2, False),            # more than 64 experts
    (64, 8, 16, 160, 96, 32, 0.1, True), (128, 8, 7, 64, 128, 32, 0.0, False), (1024, 1, 1024, 32, 64, 32, 0.0, True),
    (3, 300, 9, 64, 64, 32, 0.5, False),             # many slots a token
    (4, 2, 3, 512, 768, 256, 0.0, False),
]


@pytest.mark.parametrize("bits", [4, 3, 2])
@pytest.mark.parametrize("T,k,E,n,d,group,drop,bias", LAYERS)
def test_expert_layer(T, k, E, n, d, group, drop, bias, bits):
    ids = expert_ids(T + E, T, k, E, drop)
    r = np.random.default_rng(n + d)
    for i, (name, gated, ydt, rdt) in enumerate([("silu", True, BF16, BF16), ("gelu", False, F32, F32), ("gelu_tanh", True, F32, None),
                                                 ("none", False, BF16, F32)]):
        if (bits < 4 or T * k > 100) and i > 1:
            break
        m = 2 * d if gated else d
        up, down = fast_layers(bits + d, E, m, n, bits, group), fast_layers(bits + n, E, n, d, bits, group)
        X, w = values(n + T, T, n), r.uniform(-0.2, 1.0, (T, k)).astype(np.float32)
        b1 = r.standard_normal((E, m)).astype(np.float32) if bias else None
        b2 = r.standard_normal((E, n)).astype(np.float32) if bias else None
        res = None if rdt is None else values(7, T, n, dtype=rdt)
        wide = torch.from_numpy(np.pad(ids, ((0, 0), (0, 3)), constant_values=0)).cuda()[:, :k]
        args = (X, wide, torch.from_numpy(w).cuda(), cuda_layers(*up), cuda_layers(*down), bits, group)
        kw = dict(act=name, gated=gated, up_bias=None if b1 is None else torch.from_numpy(b1).cuda(),
                  down_bias=None if b2 is None else torch.from_numpy(b2).cuda(), residual=res)
        out = torch.full((T, n + 5), 7.0, dtype=ydt, device="cuda")
        Y = G.expert_layer(*args, out=out[:, 2:2 + n], **kw)
        x64, r64 = arr(X), None if res is None else arr(res)
        ref = L64.expert_layer(x64, ids, w, up, down, bits, group, name, gated, b1, b2, r64)
        e = layer_bound(x64, ids, w, up, down, bits, group, name, gated, b1, b2, r64, 1 if ydt == BF16 else 3)
        assert np.all(np.abs(arr(Y) - ref) <= e + last(ydt, np.abs(ref) + e))
        assert torch.all(out[:, :2] == 7) and torch.all(out[:, 2 + n:] == 7)
        assert torch.equal(G.expert_layer(*args, out_dtype=ydt, **kw), Y)


# As above: 8 groups a time in the first launch, 16 in the second, whose waves have
# all of K where the tiles are as many as they are.
LAYERS_OF_MANY_GROUPS = [
    (20, 2, 20, 128, 2432, 128, 0.0, False), (20, 2, 20, 128, 2560, 128, 0.1, True),   # 19 and 20 groups of a row
    (18, 2, 20, 64, 1312, 32, 0.0, True), (18, 2, 20, 96, 1920, 96, 0.1, False), (20, 2, 20, 64, 2688, 64, 0.0, False),
    (2, 2, 3, 4736, 128, 128, 0.0, False), (6, 2, 4, 5120, 128, 128, 0.0, True),     # 37 and 40 groups for four waves
    (1, 1, 2, 128, 34816, 128, 0.0, False),          # one tile: 272 groups for 16 or 8 waves
    (3, 300, 9, 128, 2432, 128, 0.95, False),        # more than 512 slots, eight waves
]


@pytest.mark.parametrize("bits", [4, 3, 2])
@pytest.mark.parametrize("case", LAYERS_OF_MANY_GROUPS, ids=str)
def test_expert_layer_of_many_groups_a_wave(case, bits):
    test_expert_layer(*case, bits)


def test_expert_layer_agrees_with_its_parts():
    """route, linear, linear and combine of the same tokens, and tokens that are
    dropped altogether keep their residual; the residual may be the result."""
    T, k, E, n, d, group = 24, 4, 16, 256, 128, 64
    ids = expert_ids(3, T, k, E, 0.2)
    ids[5], ids[9] = -1, E
    up, down = cuda_layers(*fast_layers(1, E, 2 * d, n, 4, group)), cuda_layers(*fast_layers(2, E, n, d, 4, group))
    X, res = values(1, T, n), values(2, T, n, dtype=F32)
    w = torch.rand(T, k, device="cuda")
    idc = torch.from_numpy(ids).cuda()
    r = G.route(idc, E)
    h = G.linear(X, *up, 4, group, act="silu", gated=True, offsets=r.offsets, rows=r.rows)
    y = G.linear(h, *down, 4, group, offsets=r.offsets, out_dtype=F32)
    want = G.combine(y, r.inverse, w) + res
    got = G.expert_layer(X, idc, w, up, down, 4, group, residual=res, out_dtype=F32)
    # h rounded to bf16 on one side: 2^-8 of the sum of magnitudes
    mag = G.combine(G.linear(h.abs(), down[0], down[1], down[2] * 0, 4, group, offsets=r.offsets, out_dtype=F32), r.inverse, w)
    assert torch.all((got - want).abs() <= 2.0 ** -8 * mag + 1e-4)
    assert torch.equal(got[5], res[5]) and torch.equal(got[9], res[9])
    assert torch.equal(G.expert_layer(X, idc, w, up, down, 4, group, residual=res, out=res), got) and torch.equal(res, got)
    empty = G.expert_layer(X[:2], idc[:2] * 0 - 1, None, up, down, 4, group)
    assert torch.count_nonzero(empty) == 0


def test_expert_layer_of_padded_ids():
    """1024 slots of which a few have an expert: LDS holds what is in use."""
    E, n, d = 6, 64, 96
    up, down = fast_layers(1, E, 2 * d, n, 4, 32), fast_layers(2, E, n, d, 4, 32)
    ids = np.full((128, 8), -1, np.int32)
    ids[77, 3], ids[127, 7] = 4, 0
    X = values(1, 128, n)
    w = np.ones((128, 8), np.float32)
    Y = arr(G.expert_layer(X, torch.from_numpy(ids).cuda(), None, cuda_layers(*up), cuda_layers(*down), 4, 32, out_dtype=F32))
    ref = L64.expert_layer(arr(X), ids, w, up, down, 4, 32, "silu", True)
    e = layer_bound(arr(X), ids, w, up, down, 4, 32, "silu", True, None, None, None, 3)
    assert np.all(np.abs(Y - ref) <= e + U32 * np.abs(ref)) and np.count_nonzero(Y.any(1)) == 2


def test_expert_layer_nonfinite_tokens_stay_apart():
    E, n, d = 4, 128, 64
    up, down = cuda_layers(*fast_layers(1, E, 2 * d, n, 4, 32)), cuda_layers(*fast_layers(2, E, n, d, 4, 32))
    X = values(1, 9, n)
    ids = torch.from_numpy(expert_ids(1, 9, 2, E)).cuda()
    want = G.expert_layer(X, ids, None, up, down, 4, 32)
    X[3, 5], X[6, 0] = float("nan"), float("inf")
    got = G.expert_layer(X, ids, None, up, down, 4, 32)
    keep = torch.tensor([0, 1, 2, 4, 5, 7, 8], device="cuda")
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[3]).all() and not torch.isfinite(got[6]).any()


@pytest.mark.parametrize("T", [1, 16])
def test_expert_layer_captured_replays(T):
    """Replayed on changing tokens and experts with eager work between; two graphs
    with workspaces of their own."""
    k, E, n, d = 4, 16, 256, 256
    up, down = cuda_layers(*fast_layers(1, E, 2 * d, n, 4, 128)), cuda_layers(*fast_layers(2, E, n, d, 4, 128))
    sets = [(values(i, T, n), torch.from_numpy(expert_ids(i, T, k, E, 0.1)).cuda(), torch.rand(T, k, device="cuda")) for i in range(3)]
    want = [G.expert_layer(*s, up, down, 4, 128) for s in sets]
    live = [t.clone() for t in sets[0]]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.expert_layer(*live, up, down, 4, 128)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(G.expert_layer(*live, up, down, 4, 128))
        graphs.append(graph)
    for i in (0, 1, 2, 1):
        for a, b in zip(live, sets[i]):
            a.copy_(b)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[i]) and torch.equal(outs[1], want[i])
        G.expert_layer(*sets[0], up, down, 4, 128)


def test_expert_layer_binding_refusals():
    E, n, d = 2, 64, 32
    up, down = cuda_layers(*fast_layers(1, E, 2 * d, n, 4, 32)), cuda_layers(*fast_layers(2, E, n, d, 4, 32))
    X, ids = values(1, 3, n), torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    G.expert_layer(X, ids, None, up, down, 4, 32)
    for bad in (lambda: G.expert_layer(X, ids[:2], None, up, down, 4, 32), lambda: G.expert_layer(X, ids, None, up, up, 4, 32),
                lambda: G.expert_layer(X, ids, torch.ones(3, 3, device="cuda"), up, down, 4, 32),
                lambda: G.expert_layer(X, ids, None, up, down, 4, 32, up_bias=torch.ones(2, 32, device="cuda")),
                lambda: G.expert_layer(X, ids, None, up, down, 4, 32, residual=X[:, :32]),
                lambda: G.expert_layer(X, ids, None, up, down, 4, 32, act="swish")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: G.expert_layer(X.float(), ids, None, up, down, 4, 32), lambda: G.expert_layer(X, ids.long(), None, up, down, 4, 32),
                lambda: G.expert_layer(X, ids, None, up, down, 4, 32, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    wide = torch.zeros(3, n + 4, dtype=BF16, device="cuda")
    many = torch.zeros(1025, 1, dtype=torch.int32, device="cuda")
    for bad in (lambda: G.expert_layer(wide[:, :n], ids, None, up, down, 4, 32),
                lambda: G.expert_layer(values(1, 1025, n), many, None, up, down, 4, 32)):
        with pytest.raises(G.GPTQError):
            bad()
    assert G.expert_layer(X[:0], ids[:0], None, up, down, 4, 32).shape == (0, n)
