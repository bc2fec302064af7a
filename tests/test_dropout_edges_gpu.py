"""The dropout operators on a B200 where values leave the ordinary range:
infinities and NaN beside finite rows and in dropped places of the gradient,
rows of the type's largest values, and a weight array off a 16-byte boundary.

The comparisons are exact wherever the definition gives an exact answer: a row
is a function of its own inputs, so a run with non-finite values in some rows
must leave the others' bits as a run without them does, and a dropped place of
dbranch is zero whatever stands in dx."""
import numpy as np
import pytest
import torch

import dropout_ref as dr
import gpu_util as gu
import oracle
import tolerances as tol

pytestmark = pytest.mark.gpu

RECOMPUTE = 4
SEED, OFFSET, P, EPS = 99, 1 << 33, 0.25, 1e-5

# rows of several per warp, whole vectors and not, one warp, several warps, the
# rings, the split ring, past them (16 bits) and past the ragged kernels
WIDTHS = [12, 64, 601, 768, 1024, 1031, 1600, 2048, 6145, 8193, 12296]


@pytest.fixture(scope="module")
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return gu.ln()


def _rows(C, many):
    """Few rows: the one-launch backward where there is one; many: a grid that
    takes several turns where the rows are short, the last with groups of a
    warp that have no row."""
    return 7 if not many else (20009 if C <= 64 else 1203 if C <= 2048 else 67)


def _normal(gen, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(gu.TORCH_DT[dtype])


def _kept(N, C):
    return torch.from_numpy(dr.keep(N * C, P, SEED, OFFSET).reshape(N, C)).cuda()


def _forward(lib, dtype, resid, branch, w, b, p=P):
    N, C = resid.shape
    x = gu.nan_tensor((N, C), resid.dtype)
    out, mean, rstd = gu.forward_outputs(N, C, dtype)
    lib.ln_forward_dropout_residual(x, out, mean, rstd, resid, branch, w, b, N, C, EPS, p, SEED,
                                    OFFSET, None, gu.DT[dtype])
    return x, out, mean, rstd


def _backward(lib, dtype, inp, dout, w, stats, prev, inplace=False, p=P):
    """stats: (mean, rstd), or None to recompute them."""
    N, C = inp.shape
    dres, dbr = (gu.nan_tensor((N, C), inp.dtype) for _ in range(2))
    dw, db = (gu.nan_tensor((C,), torch.float32) for _ in range(2))
    if inplace:
        dres.copy_(prev)
        prev = dres
    mean, rstd = stats or (None, None)
    lib.ln_backward_dropout_residual(dres, dbr, dw, db, prev, dout, inp, w, mean, rstd, N, C, EPS,
                                     p, SEED, OFFSET, None, gu.DT[dtype],
                                     0 if stats else RECOMPUTE)
    return dres, dbr, dw, db


def _same_bits(name, a, b, rows=None):
    a, b = (a, b) if rows is None else (a[rows], b[rows])
    bad = gu.bits(a.contiguous()) != gu.bits(b.contiguous())
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} differ"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("many", [False, True])
def test_non_finite_rows_stay_alone(lib, dtype, C, many):
    """Infinities and NaN in three rows (resid, branch, inp or dout; with rows
    that share a 16-byte vector with their neighbours): the other rows' results
    are those of a run without them, bit for bit."""
    N = _rows(C, many)
    g = torch.Generator(device="cuda").manual_seed(N + C)
    w, b = 1 + _normal(g, (C,), dtype, 0.1), _normal(g, (C,), dtype, 0.1)
    resid, branch, dout, prev = (_normal(g, (N, C), dtype) for _ in range(4))
    bad = torch.tensor([1, N // 2, N - 1], device="cuda")
    fine = torch.ones(N, dtype=torch.bool, device="cuda")
    fine[bad] = False
    clean = _forward(lib, dtype, resid, branch, w, b)
    r2, b2 = resid.clone(), branch.clone()
    r2[bad[0]] = float("inf")
    b2[bad[1]] = float("nan")
    r2[bad[2], ::2] = float("-inf")
    b2[bad[2], 1::2] = float("inf")
    for name, u, v in zip(("x", "out", "mean", "rstd"), clean, _forward(lib, dtype, r2, b2, w, b)):
        assert torch.isfinite(u).all()
        _same_bits(f"{dtype} {N}x{C} {name}", u, v, fine)

    x, _, mean, rstd = clean
    for stats in ((mean, rstd), None):
        for inplace in (False, True):
            ref = _backward(lib, dtype, x, dout, w, stats, prev, inplace)
            x2, d2 = x.clone(), dout.clone()
            x2[bad[0]] = float("inf")
            d2[bad[1]] = float("nan")
            x2[bad[2], ::2] = float("nan")
            d2[bad[2], 1::2] = float("-inf")
            got = _backward(lib, dtype, x2, d2, w, stats, prev, inplace)
            for name, u, v in zip(("dresid", "dbranch"), ref, got):
                assert torch.isfinite(u).all()
                _same_bits(f"{dtype} {N}x{C} {name} saved={stats is not None}", u, v, fine)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("many", [False, True])
def test_dbranch_is_zero_where_dropped(lib, dtype, C, many):
    """Infinities and NaN of the gradient in dropped places leave exact zeros in
    dbranch, come through in kept places, and touch neither the other elements
    nor dweight and dbias (dresid_out enters no sum)."""
    N = _rows(C, many)
    g = torch.Generator(device="cuda").manual_seed(3 * N + C)
    w = 1 + _normal(g, (C,), dtype, 0.1)
    x, dout, prev = (_normal(g, (N, C), dtype) for _ in range(3))
    _, mean, rstd = gu.forward(lib, x, w, w, N, C, EPS, dtype)
    kept = _kept(N, C)
    p2 = prev.clone()
    p2[:, 0::3] = float("nan")
    p2[:, 1::3] = float("-inf")
    hurt = torch.zeros(C, dtype=torch.bool, device="cuda")
    hurt[0::3] = hurt[1::3] = True
    for stats in ((mean, rstd), None):
        for inplace in (False, True):
            label = f"{dtype} {N}x{C} saved={stats is not None} inplace={inplace}"
            ref = _backward(lib, dtype, x, dout, w, stats, prev, inplace)
            dres, dbr, dw, db = _backward(lib, dtype, x, dout, w, stats, p2, inplace)
            assert (dbr[~kept] == 0).all(), f"{label}: dropped places"
            assert not torch.isfinite(dbr[:, hurt][kept[:, hurt]]).any(), label
            assert not torch.isfinite(dres[:, hurt]).any(), label
            _same_bits(f"{label} dresid", dres[:, ~hurt], ref[0][:, ~hurt])
            _same_bits(f"{label} dbranch", dbr[:, ~hurt], ref[1][:, ~hurt])
            _same_bits(f"{label} dweight", dw, ref[2])
            _same_bits(f"{label} dbias", db, ref[3])
            # a rate of one: nothing reaches the branch
            _, none, _, _ = _backward(lib, dtype, x, dout, w, stats, p2, inplace, p=1.0)
            assert (none == 0).all(), f"{label}: p = 1"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("many", [False, True])
def test_rows_of_the_largest_values(lib, dtype, C, many):
    """The odd rows (few rows: every row) a constant of the type's lowest
    value.  x - mean is then exactly zero: out is bias, rstd 1 / sqrt(eps),
    xhat zero, dresid and dbranch and the column sums finite and those of the
    definition."""
    N = _rows(C, many)
    g = torch.Generator(device="cuda").manual_seed(5 * N + C)
    low = torch.finfo(gu.TORCH_DT[dtype]).min
    w, b = 1 + _normal(g, (C,), dtype, 0.1), _normal(g, (C,), dtype, 0.1)
    resid, dout, prev = (_normal(g, (N, C), dtype) for _ in range(3))
    resid[1::2 if many else 1] = low
    resid[0] = low
    branch = torch.zeros_like(resid)
    x, out, mean, rstd = _forward(lib, dtype, resid, branch, w, b)
    label = f"{dtype} {N}x{C}"
    _same_bits(f"{label} x", x, resid)
    flat = (resid == low).all(1)
    _same_bits(f"{label} out", out[flat], b.expand(int(flat.sum()), C))
    assert (mean[flat] == low).all(), f"{label}: mean {mean[flat][:4]}"
    kept = dr.keep(N * C, P, SEED, OFFSET).reshape(N, C)
    h = gu.to_f64
    _, m64, s64 = oracle.default().forward(h(x), h(w), h(b), EPS)
    tol.check(f"{label} rstd", h(rstd), s64, dtype, "stats")
    m32, s32 = m64.astype(np.float32), s64.astype(np.float32)
    for saved in (True, False):
        stats = (torch.from_numpy(m32).cuda(), torch.from_numpy(s32).cuda()) if saved else None
        got = _backward(lib, dtype, x, dout, w, stats, prev)
        ref = dr.backward(h(prev), h(dout), h(x), h(w), m32, s32, EPS, kept, P, not saved)
        sc = tol.magnitude_scales(h(x), h(dout), h(w), m64, s64)
        up = float(dr.scale32(P))
        for name, kind, u, v, s in zip(
                ("dresid", "dbranch", "dweight", "dbias"),
                ("act_bwd", "act_bwd", "param_grad", "param_grad"), got, ref,
                (sc["dinp"], sc["dinp"] * up, sc["dweight"], sc["dbias"])):
            assert torch.isfinite(u).all(), f"{label} {name} saved={saved}: not finite"
            tol.check(f"{label} {name} saved={saved}", h(u), v, dtype, kind, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", WIDTHS)
def test_mean_of_a_row_with_an_infinity(lib, dtype, C):
    """mean is the sum of the row over C: infinite where the row holds an
    infinity of one sign (in a kept place, not the first, which is the point the
    distances are taken from), as ln_forward gives it for the stored row."""
    N = 6
    g = torch.Generator(device="cuda").manual_seed(C)
    w, b = 1 + _normal(g, (C,), dtype, 0.1), _normal(g, (C,), dtype, 0.1)
    resid, branch = (_normal(g, (N, C), dtype) for _ in range(2))
    resid[1, C // 2] = float("inf")
    resid[2, C - 1] = float("-inf")
    x, _, mean, rstd = _forward(lib, dtype, resid, branch, w, b)
    _, m2, r2 = gu.forward(lib, x, w, b, N, C, EPS, dtype)
    assert mean[1] == float("inf") and mean[2] == float("-inf"), mean
    assert torch.equal(torch.isnan(mean), torch.isnan(m2))
    assert torch.isnan(rstd[1:3]).all() and torch.isnan(r2[1:3]).all()
    assert torch.isfinite(mean[[0, 3, 4, 5]]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("many", [False, True])
def test_weight_off_a_boundary(lib, dtype, C, many):
    """weight and bias that start one element into an allocation, everything
    else on 16 bytes: what aligned copies of them give, to the tolerances of
    the two kernels that may serve the calls."""
    N = _rows(C, many)
    g = torch.Generator(device="cuda").manual_seed(7 * N + C)
    w, b = 1 + _normal(g, (C + 1,), dtype, 0.1), _normal(g, (C + 1,), dtype, 0.1)
    w, b = w[1:], b[1:]
    assert w.data_ptr() % 16 == gu.SIZE[dtype] == b.data_ptr() % 16
    wa, ba = w.clone(), b.clone()
    resid, branch, dout, prev = (_normal(g, (N, C), dtype) for _ in range(4))
    label = f"{dtype} {N}x{C}"
    ref = _forward(lib, dtype, resid, branch, wa, ba)
    got = _forward(lib, dtype, resid, branch, w, b)
    _same_bits(f"{label} x", got[0], ref[0])
    h = gu.to_f64
    rout, m64, s64 = oracle.default().forward(h(got[0]), h(w), h(b), EPS)
    sc = tol.magnitude_scales(h(got[0]), h(dout), h(w), m64, s64)
    tol.check(f"{label} out", h(got[1]), rout, dtype, "act_fwd")
    tol.check(f"{label} mean", h(got[2]), m64, dtype, "stats", sc["mean"])
    tol.check(f"{label} rstd", h(got[3]), s64, dtype, "stats")
    kept = dr.keep(N * C, P, SEED, OFFSET).reshape(N, C)
    m32, s32 = m64.astype(np.float32), s64.astype(np.float32)
    for saved in (True, False):
        stats = (torch.from_numpy(m32).cuda(), torch.from_numpy(s32).cuda()) if saved else None
        grads = _backward(lib, dtype, got[0], dout, w, stats, prev)
        want = dr.backward(h(prev), h(dout), h(got[0]), h(w), m32, s32, EPS, kept, P, not saved)
        up = float(dr.scale32(P))
        for name, kind, u, v, s in zip(
                ("dresid", "dbranch", "dweight", "dbias"),
                ("act_bwd", "act_bwd", "param_grad", "param_grad"), grads, want,
                (sc["dinp"], sc["dinp"] * up, sc["dweight"], sc["dbias"])):
            tol.check(f"{label} {name} saved={saved}", h(u), v, dtype, kind, s)
    assert lib.device_status() == 0


def _counter(kind):
    return {"int32": lambda: torch.zeros(2, dtype=torch.int32, device="cuda"),
            "float64": lambda: torch.ones(1, dtype=torch.float64, device="cuda"),
            "complex64": lambda: torch.ones(1, dtype=torch.complex64, device="cuda"),
            "two": lambda: torch.zeros(2, dtype=torch.int64, device="cuda"),
            "none": lambda: torch.zeros(0, dtype=torch.int64, device="cuda"),
            "host": lambda: torch.zeros(1, dtype=torch.int64)}[kind]()


@pytest.mark.parametrize("kind", ["int32", "float64", "complex64", "two", "none", "host"])
def test_other_counters_are_refused(lib, kind):
    """step is one 64-bit integer of the current GPU; anything else is refused
    by every call before a kernel runs."""
    step = _counter(kind)
    N, C = 4, 8
    a = [torch.zeros(N, C, device="cuda") for _ in range(6)]
    v = [torch.ones(C, device="cuda") for _ in range(4)]
    n0 = lib.launch_count()
    with pytest.raises(TypeError):
        lib.ln_dropout(a[0], a[1], N * C, P, 0, 0, step, lib.LN_F32)
    with pytest.raises(TypeError):
        lib.ln_forward_dropout_residual(a[0], a[1], v[0], v[1], a[2], a[3], v[2], v[3], N, C, EPS,
                                        P, 0, 0, step, lib.LN_F32)
    with pytest.raises(TypeError):
        lib.ln_backward_dropout_residual(a[0], a[1], v[0], v[1], None, a[2], a[3], v[2], v[3],
                                         v[3], N, C, EPS, P, 0, 0, step, lib.LN_F32)
    assert lib.launch_count() == n0


def test_integer_counters_are_taken(lib):
    """int64 and uint64, of one element and of any number of dimensions, an
    element of a larger tensor too: all draw the same mask."""
    n = 4096
    inp = torch.ones(n, device="cuda")
    base = torch.tensor([3, 7, 11], dtype=torch.int64, device="cuda")
    want = dr.keep(n, P, SEED, OFFSET, 7)
    for step in (base[1], base[1:2], base[1].reshape(1, 1), base[1:2].view(torch.uint64),
                 base.data_ptr() + 8):
        out = torch.empty_like(inp)
        lib.ln_dropout(out, inp, n, P, SEED, OFFSET, step, lib.LN_F32)
        assert np.array_equal(gu.to_f64(out) != 0, want)
