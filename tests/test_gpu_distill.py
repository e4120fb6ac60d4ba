"""Distillation from a teacher's top logits on the GPU against the float64
oracle (oracle/layers.py), through the C ABI.

Tolerances, with u = 2^-24 (half a step of fp32, relative) and 2^-8 for bf16:
 * The sum of V exponentials: each exponent (z - m) / tau is off by 3 u of its
   magnitude (difference, factor, product), the exponential by 2 u more; rescaled
   sums and at most V additions of positive values: l is off by
   (3 A + 4 + depth) u relatively, where A is the largest exponent that counts
   (terms below exp(-A) of the largest add less than u for A = 30), and depth
   the additions in one chain, at most V / 256 + 64 (one row's threads are 256
   or 1024). lse: that, plus 4 u of its own magnitude and of m / tau.
 * p: exponents off by 4 u of their magnitude P, sums of K terms: (4 P + K / 256 +
   20) u relatively; log p: 4 u (P + log K + 1).
 * loss: sum over p (log p - log q) of the factors' errors, and K / 256 + 16
   additions.
 * dZ: q's exponent is off by u of itself, by u |z / tau| and by lse's error.
"""
import numpy as np
import pytest

from oracle import layers as L64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import post_weight_quantization_28_amd as G  # noqa: E402

U32, UBF = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


def arr(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(seed, T, V, K, logp, dtype, scale=3.0):
    r = np.random.default_rng(seed)
    Z = torch.from_numpy((scale * r.standard_normal((T, V))).astype(np.float32)).to(dtype)
    ids = np.stack([r.choice(V, K, replace=K > V) for _ in range(T)]).astype(np.int32).reshape(T, K)
    teacher = (2.0 * r.standard_normal((T, K))).astype(np.float32)
    if logp:
        teacher = (teacher - np.log(np.exp(teacher.astype(np.float64)).sum(1, keepdims=True)) - 0.2).astype(np.float32)
    gone = r.random((T, K)) < 0.1
    ids[gone] = np.where(r.random(int(gone.sum())) < 0.5, -1, V)     # both sides of the range
    grad = r.uniform(0.2, 1.5, T).astype(np.float32)
    return Z, ids, teacher, grad


def bounds(Z, ids, teacher, temp, logp, loss, lse, ps, grad, dref):
    """Absolute bounds on (loss, lse, dZ) by the count above, dZ before its last rounding."""
    T, V = Z.shape
    K = ids.shape[1]
    s = Z / temp
    big = np.abs(np.where(np.isfinite(s), s, 0.0)).max(1)
    depth = V / 256 + 64
    e_lse = U32 * (3 * 30 + 4 + depth + 4 * (np.abs(lse) + big))
    P = np.abs(np.where(np.isfinite(teacher), teacher, 0.0)).max() * 2 / (1.0 if logp else temp)
    rel_p = U32 * (4 * P + K / 256 + 20)
    abs_lp = U32 * 4 * (P + np.log(K) + 1)
    e_loss = np.zeros(T)
    for t in range(T):
        for v, p in ps[t]:
            if p > 0:
                term = abs(np.log(p)) + abs(s[t, v] - lse[t])
                e_loss[t] += p * ((rel_p + (K / 256 + 16) * U32) * term + abs_lp + e_lse[t] + 4 * U32 * (big[t] + abs(s[t, v])))
    e_d = np.zeros((T, V))
    for t in range(T):
        mass = sum(p for _, p in ps[t])
        if mass == 0:
            continue
        with np.errstate(invalid="ignore"):
            arg = np.where(np.isfinite(s[t]), np.abs(s[t] - lse[t]), 0.0)
            q = np.exp(s[t] - lse[t])
        f = abs(grad[t]) / temp
        e_d[t] = f * mass * q * (U32 * (3 * arg + big[t] + 10) + rel_p + e_lse[t])
        for v, p in ps[t]:
            e_d[t, v] += f * p * (rel_p + (K + 4) * U32)
        e_d[t] += 4 * U32 * np.abs(dref[t])
    return e_loss, e_lse, e_d


def check(Z, ids, teacher, grad, temp, logp, odt, out=None):
    Zc, idc, tc, gc = Z.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda(), torch.from_numpy(grad).cuda()
    z64 = arr(Z)
    loss, lse, ps = L64.distill(z64, ids, teacher, temp, logp)
    ref = L64.distill_grad(z64, lse, ps, grad, temp)
    e_loss, e_lse, e_d = bounds(z64, ids, teacher, temp, logp, loss, lse, ps, grad, ref)
    a, b = G.distill(Zc, idc, tc, temperature=temp, log_probs=logp)
    assert np.all(np.abs(arr(b) - lse) <= e_lse)
    assert np.all(np.abs(arr(a) - loss) <= e_loss)
    d = G.distill_grad(Zc, idc, tc, b, gc, temperature=temp, log_probs=logp, out_dtype=odt)
    tol = e_d + ((UBF * (np.abs(ref) + e_d) + 2.0 ** -134) if d.dtype == BF16 else 2.0 ** -126)
    assert np.all(np.abs(arr(d) - ref) <= tol)
    again = G.distill(Zc, idc, tc, temperature=temp, log_probs=logp)
    assert torch.equal(again[0], a) and torch.equal(again[1], b)
    same = Zc.clone()
    if d.dtype == Z.dtype:                                            # in place
        G.distill_grad(same, idc, tc, b, gc, temperature=temp, log_probs=logp, out=same)
        assert torch.equal(same, d)
    return a, b, d


CASES = [   # T, V, K, temperature, log probabilities
    (1, 1, 1, 1.0, False), (1, 7, 3, 2.0, True), (3, 8, 8, 1.0, False), (5, 9, 4, 0.5, False), (2, 255, 17, 1.0, True),
    (4, 2047, 300, 4.0, False), (7, 2049, 64, 1.0, False), (3, 8193, 256, 3.0, True),     # 1024 threads, parts of the gradient's
    (1, 50001, 1, 1.0, False), (2, 33333, 1024, 1.0, True), (1030, 1000, 5, 2.0, False),  # 256 threads a row
    (1024, 2304, 2, 1.0, False), (40, 5000, 257, 1.5, False),
]


@pytest.mark.parametrize("zdt,odt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T,V,K,temp,logp", CASES)
def test_distill(T, V, K, temp, logp, zdt, odt):
    check(*inputs(T + V + K, T, V, K, logp, zdt), temp, logp, odt)


def test_padding_rows_give_zero_whatever_they_hold():
    """No entry, no mass, or a teacher of -infinity: loss 0 and gradient 0,
    also where the logits are NaN."""
    for V, T in ((300, 5), (9000, 5), (700, 1100)):
        Z, ids, teacher, grad = inputs(V, T, V, 4, False, F32)
        ids[0], ids[1], teacher[2] = -1, V + 3, -np.inf
        Z[0, 5] = float("nan")
        Z[1] = float("-inf")
        Zc, args = Z.cuda(), (torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda())
        loss, lse = G.distill(Zc, *args)
        d = G.distill_grad(Zc, *args, lse, torch.from_numpy(grad).cuda())
        assert torch.count_nonzero(loss[:3]) == 0 and torch.count_nonzero(d[:3]) == 0
        assert torch.isfinite(loss).all() and torch.isfinite(d).all() and torch.all(loss[3:] != 0)
        assert torch.isnan(lse[0]) and lse[1] == float("-inf")


def test_masked_entries_and_lowest_values():
    """Logits of -infinity have no probability, the type's lowest value is a
    logit like another, NaN and +infinity spoil their own row only."""
    for zdt in (BF16, F32):
        low = torch.finfo(zdt).min
        for V in (100, 20000):
            Z, ids, teacher, grad = inputs(V, 6, V, 6, False, zdt)
            ids[:] = np.arange(6) * 7 + 1
            Z[0, 50:] = float("-inf")
            Z[1, 50:] = low
            Z[2] = low                                     # every entry alike: a uniform distribution
            Z[3, 60] = float("nan")
            Z[4, 60] = float("inf")
            Zc, idc, tc = Z.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda()
            loss, lse = G.distill(Zc, idc, tc)
            z64 = arr(Z[[0, 1, 5]])
            with np.errstate(over="ignore"):
                l64, e64, ps = L64.distill(z64, ids[[0, 1, 5]], teacher[[0, 1, 5]], 1.0, False)
                ref = L64.distill_grad(z64, e64, ps, grad[[0, 1, 5]], 1.0)
            keep = torch.tensor([0, 1, 5])
            d = G.distill_grad(Zc, idc, tc, lse, torch.from_numpy(grad).cuda(), out_dtype=F32)
            # exponents up to 40: 3 40 u and the sums' V / 256 + 64 additions, lse's own rounding 4 20 u
            e = U32 * (120 + V / 256 + 64 + 80)
            assert np.all(np.abs(arr(lse)[keep] - e64) <= e) and np.all(np.abs(arr(loss)[keep] - l64) <= 2 * e)
            assert np.all(np.abs(arr(d)[keep] - ref) <= 2 * e * grad[[0, 1, 5]][:, None])
            assert torch.count_nonzero(d[:2, 50:]) == 0
            p = np.exp(teacher[2].astype(np.float64) - teacher[2].max())
            p /= p.sum()
            assert abs(float(loss[2]) - (float((p * np.log(p)).sum()) + np.log(V))) <= 2 * e
            assert torch.isnan(loss[3]) and torch.isnan(loss[4])
            one = ids[5:6].copy()                          # the teacher's entry is masked: an infinite loss, a finite gradient
            Zm = Z[5:6].clone()
            Zm[0, one[0, 0]] = float("-inf")
            lo, le = G.distill(Zm.cuda(), torch.from_numpy(one).cuda(), tc[5:6])
            dd = G.distill_grad(Zm.cuda(), torch.from_numpy(one).cuda(), tc[5:6], le, torch.ones(1).cuda())
            assert lo[0] == float("inf") and torch.isfinite(dd).all()
            tm = tc[5:6].clone()
            tm[0, 0] = float("-inf")                       # unless the teacher has no mass there
            assert torch.isfinite(G.distill(Zm.cuda(), torch.from_numpy(one).cuda(), tm)[0]).all()


@pytest.mark.parametrize("temp", [1.0, 0.02])
@pytest.mark.parametrize("T,V", [(6, 100), (6, 20000), (1100, 2500)])   # one part a row, several, one of many rows
def test_gradient_far_from_zero(T, V, temp):
    """Rows whose lse is far from zero, where fp32's lse says little about the sum:
    lowest values everywhere (uniform), in half of a row, large offsets, a low
    temperature. Against the oracle on the logits less their largest, which changes
    neither loss nor gradient. An exponent x = (z - m) / tau - log l is off by 6 u of
    |x| + 2 log V (difference, tau, 1 / tau, fused product, log2 e, product; log l),
    the exponential and its factors by 8 u, l as counted above; near rows
    (|lse| <= 128, with a bf16 dZ 2048) by lse's error instead."""
    for zdt in (BF16, F32):
        low = torch.finfo(zdt).min
        Z, ids, teacher, grad = inputs(V, T, V, 6, False, zdt)
        ids[:] = np.arange(6) * 7 + 1
        Z[0] = low
        Z[1] += 1e4
        Z[2] -= 1e5
        Z[3, V // 2:] = low
        Z[4] *= 1e3
        z64 = arr(Z)
        near = np.abs(L64.distill(z64, ids, teacher, temp, False)[1])
        big = np.abs(z64).max(1) / temp
        zs = z64 - z64.max(1, keepdims=True)
        loss, lse, ps = L64.distill(zs, ids, teacher, temp, False)
        ref = L64.distill_grad(zs, lse, ps, grad, temp)
        x = np.abs(zs) / temp
        f = (grad / temp)[:, None]
        P = 2 * np.abs(teacher).max() / temp
        rel_p = U32 * (4 * P + 6 / 256 + 20)
        args = (torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda())
        Zc, gc = Z.cuda(), torch.from_numpy(grad).cuda()
        le = G.distill(Zc, *args, temperature=temp)[1]
        for odt in (BF16, F32):
            rel = 6 * (x + 2 * np.log(V)) + 8 + 3 * 30 + 4 + V / 256 + 64
            rel += np.where(near <= (2048 if odt == BF16 else 128), 4 * (near + big), 0)[:, None]
            e = (np.exp(-x - lse[:, None]) * (U32 * rel + rel_p) + 4 * U32 * np.abs(ref)) * f
            e[:, ids[0]] += f * np.array([[p for _, p in row] for row in ps]) * (rel_p + 10 * U32)
            # q below 2^-126, the smallest normal number, is 0 (the exponential has no subnormal results), which the
            # factor grad / tau makes up to grad / tau 2^-126 of dZ (at tau = 0.02 2.7e-40 of an fp32 row 1 became 0)
            e += f * 2.0 ** -126
            d = G.distill_grad(Zc, *args, le, gc, temperature=temp, out_dtype=odt)
            tol = e + ((UBF * (np.abs(ref) + e) + 2.0 ** -134) if odt == BF16 else U32 * np.abs(ref) + 2.0 ** -126)
            assert np.all(np.abs(arr(d) - ref) <= tol)
            if odt == zdt:
                same = Zc.clone()
                G.distill_grad(same, *args, le, gc, temperature=temp, out=same)
                assert torch.equal(same, d)


def test_repeated_ids_count_each_time():
    Z, ids, teacher, grad = inputs(5, 3, 4100, 600, True, F32)
    ids[:, ::2] = 17
    ids[:, 5] = 2048
    teacher -= 1.0
    check(Z, ids, teacher, grad, 1.0, True, F32)


def test_pitches_and_untouched_columns():
    """Rows apart and unaligned: same results, and nothing beside them is written."""
    for zdt in (BF16, F32):
        Z, ids, teacher, grad = inputs(9, 5, 4099, 33, False, zdt)
        a, b, d = check(Z, ids, teacher, grad, 2.0, False, zdt)
        wide = torch.full((5, 4110), 7.0, dtype=zdt, device="cuda")
        wide[:, 3:4102] = Z.cuda()
        args = (torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda())
        x, y = G.distill(wide[:, 3:4102], *args, temperature=2.0)
        assert torch.equal(x, a) and torch.equal(y, b)
        out = torch.full((5, 4107), 9.0, dtype=zdt, device="cuda")
        G.distill_grad(wide[:, 3:4102], *args, y, torch.from_numpy(grad).cuda(), temperature=2.0, out=out[:, 5:4104])
        assert torch.equal(out[:, 5:4104], d) and torch.all(out[:, :5] == 9) and torch.all(out[:, 4104:] == 9)


def test_gradient_against_differences():
    """Central differences of the fp64 loss at the GPU's gradient, and the
    gradient's sum: M q sums to M, so each row's gradient sums to 0."""
    Z, ids, teacher, grad = inputs(3, 3, 40, 6, False, F32, scale=1.0)
    idc, tc, gc = torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda(), torch.from_numpy(grad).cuda()
    loss, lse = G.distill(Z.cuda(), idc, tc, temperature=2.0)
    d = arr(G.distill_grad(Z.cuda(), idc, tc, lse, gc, temperature=2.0))
    z = arr(Z)
    h = 1e-4
    for t in range(3):
        for v in range(40):
            up, dn = z.copy(), z.copy()
            up[t, v] += h
            dn[t, v] -= h
            diff = (L64.distill(up, ids, teacher, 2.0, False)[0][t] - L64.distill(dn, ids, teacher, 2.0, False)[0][t]) / (2 * h)
            # differences: third derivative (at most 1 / tau^3) h^2 / 6, and 64-bit rounding over h; gradient: 100 u
            assert abs(d[t, v] - grad[t] * diff) <= grad[t] * (h * h + 1e-11 + 100 * U32)
    assert np.all(np.abs(d.sum(1)) <= 100 * U32 * grad)


def test_rows_beyond_32_bits():
    """Logits whose offsets pass 2^32 bytes and 2^31 values: the last rows agree with the same rows alone."""
    T, V = 16500, 131101
    Z = torch.empty(T, V, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for lo in range(0, T, 4125):
        Z[lo:lo + 4125] = torch.randn(4125, V, generator=g, device="cuda")
    ids = torch.randint(0, V, (T, 3), generator=g, device="cuda").to(torch.int32)
    teacher = torch.randn(T, 3, generator=g, device="cuda")
    grad = torch.rand(T, generator=g, device="cuda")
    loss, lse = G.distill(Z, ids, teacher)
    part = slice(T - 1100, T)                              # enough rows for the same code
    l2, e2 = G.distill(Z[part].clone(), ids[part], teacher[part])
    assert torch.equal(loss[part], l2) and torch.equal(lse[part], e2)
    d2 = G.distill_grad(Z[part].clone(), ids[part], teacher[part], e2, grad[part])
    G.distill_grad(Z, ids, teacher, lse, grad, out=Z)
    assert torch.equal(Z[part], d2)


@pytest.mark.parametrize("T", [3, 1100])
def test_captured_step_replays(T):
    """Loss and gradient in a captured graph, replayed with eager work between:
    bitwise the eager result."""
    V, K = 5003, 16
    Z, ids, teacher, grad = inputs(T, T, V, K, False, BF16)
    Zc, idc, tc, gc = Z.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda(), torch.from_numpy(grad).cuda()
    want = {}
    for i in range(3):
        zi = (Zc.float() * (1.0 + i)).to(BF16)
        loss, lse = G.distill(zi, idc, tc)
        want[i] = (loss, lse, G.distill_grad(zi, idc, tc, lse, gc))
    live = Zc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss, lse = G.distill(live, idc, tc)
        G.distill_grad(live, idc, tc, lse, gc)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = G.distill(live, idc, tc)
        d = G.distill_grad(live, idc, tc, lse, gc)
    for i in (0, 1, 2, 1, 0):
        live.copy_((Zc.float() * (1.0 + i)).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[i][0]) and torch.equal(lse, want[i][1]) and torch.equal(d, want[i][2])
        G.distill(Zc, idc, tc)


def test_two_streams_at_once():
    """Calls on two streams do not meet."""
    sets = [inputs(s, 4, 40000, 8, False, F32) for s in (1, 2)]
    want = []
    for Z, ids, teacher, grad in sets:
        want.append(G.distill(Z.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda()))
    dev = [(Z.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(teacher).cuda()) for Z, ids, teacher, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(G.distill(*dev[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in got[i]:
            assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])


def test_binding_refusals():
    Z = torch.zeros(4, 10, dtype=BF16, device="cuda")
    ids, t, v = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda"), torch.zeros(4, device="cuda")
    for bad in (lambda: G.distill(Z.half(), ids, t), lambda: G.distill(Z, ids.long(), t), lambda: G.distill(Z, ids, t.to(BF16)),
                lambda: G.distill(Z, None, t), lambda: G.distill_grad(Z, ids, t, None, v),
                lambda: G.distill_grad(Z, ids, t, v, v, out_dtype=torch.float16)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: G.distill(Z, ids[:3], t), lambda: G.distill(Z, ids, t[:, :1]), lambda: G.distill(Z[0], ids, t),
                lambda: G.distill_grad(Z, ids, t, v[:3], v), lambda: G.distill_grad(Z, ids, t, v, v, out=Z[:, :9])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: G.distill(Z, ids, t, temperature=0.0), lambda: G.distill(Z, ids, t, temperature=float("nan")),
                lambda: G.distill(Z, ids[:, :0].contiguous(), t[:, :0].contiguous())):
        with pytest.raises(G.GPTQError):
            bad()
    loss, lse = G.distill(Z[:0], ids[:0], t[:0])
    assert loss.shape == (0,) and G.distill_grad(Z[:0], ids[:0], t[:0], lse, v[:0]).shape == (0, 10)
