"""Host-side checks of the operators over rows of logits and of the microscaled 4-bit
floats: their oracles against closed forms, brute force and differences, and the
refusals of the C ABI and of the binding (CPU only: no kernel is launched)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import weight_quantization_aware_b200 as eqat
from oracle import fp4, rows

OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, WS = range(7)
FAKE = 0x100  # aligned, never dereferenced


def P(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    from weight_quantization_aware_b200 import build
    build.build()
    return eqat.load_library()


# ------------------------------------------------------------------ oracles


def test_logprobs_oracle_closed_forms():
    x = np.log(np.array([[1.0, 2.0, 5.0], [1.0, 1.0, 1.0]]))
    lp, ent, ids, top = rows.token_logprobs(x, np.array([2, -1]), 2)
    assert np.isclose(lp[0], np.log(5 / 8)) and lp[1] == 0
    p = np.array([1, 2, 5]) / 8
    assert np.isclose(ent[0], -(p * np.log(p)).sum()) and np.isclose(ent[1], np.log(3))
    assert ids.tolist() == [[2, 1], [0, 1]]
    assert np.allclose(top[0], np.log([5 / 8, 2 / 8]))
    # a temperature is a power of the masses
    lp2, *_ = rows.token_logprobs(x, np.array([2, 0]), 0, 0.5)
    assert np.isclose(lp2[0], np.log(25 / 30))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0])
def test_distill_oracle_gradient_matches_differences(tail, tau):
    """Central differences of the loss in fp64: error of order h^2 plus 2^-52 / h."""
    rng = np.random.default_rng(5)
    T, V, k = 4, 23, 5
    x = rng.normal(size=(T, V))
    x[1, 7] = -np.inf
    ids = np.stack([rng.permutation(V)[:k] for _ in range(T)])
    ids[2, 3] = -1
    ids[3, 1] = ids[3, 0]  # an id given twice
    ids[1][ids[1] == 7] = 8
    tlp = np.log(rng.dirichlet(np.ones(k + 1), size=T)[:, :k])
    w = np.array([1.0, 0.5, 2.0, 1.5])
    loss, grad = rows.distill_topk(x, ids, tlp, w, tau, tail)
    h = 1e-5
    for t, j in itertools.product(range(T), range(V)):
        if x[t, j] == -np.inf:
            assert grad[t, j] == 0
            continue
        up, dn = x.copy(), x.copy()
        up[t, j] += h
        dn[t, j] -= h
        d = (rows.distill_topk(up, ids, tlp, w, tau, tail)[0][t] - rows.distill_topk(dn, ids, tlp, w, tau, tail)[0][t]) / (2 * h)
        assert abs(d - grad[t, j]) < 1e-8
    assert (loss > 0).all()
    assert np.abs(grad.sum(1)).max() < 1e-12  # the loss does not change when a row is shifted


@pytest.mark.parametrize("tail", [False, True])
def test_distill_oracle_ignores_what_an_empty_slot_holds(tail):
    rng = np.random.default_rng(8)
    x, ids = rng.normal(size=(5, 30)), np.tile(np.arange(4), (5, 1))
    tlp = np.log(rng.dirichlet(np.ones(5), size=5)[:, :4])
    ids[:, 2] = -1
    want = rows.distill_topk(x, np.delete(ids, 2, 1), np.delete(tlp, 2, 1), None, 1.0, tail)
    tlp[:, 2] = [np.nan, np.inf, -np.inf, 0.0, 1e30]
    for a, b in zip(rows.distill_topk(x, ids, tlp, None, 1.0, tail), want):
        assert np.array_equal(a, b) and np.isfinite(a).all()


def test_distill_oracle_is_zero_at_the_teacher():
    rng = np.random.default_rng(6)
    x = rng.normal(size=(3, 40))
    _, _, ids, tlp = rows.token_logprobs(x, np.zeros(3, int), 40, 1.5)
    loss, grad = rows.distill_topk(x, ids, tlp, None, 1.5, False)
    assert np.abs(loss).max() < 1e-12 and np.abs(grad).max() < 1e-12
    loss, grad = rows.distill_topk(x, ids[:, :6], tlp[:, :6], None, 1.5, True)
    assert np.abs(loss).max() < 1e-12 and np.abs(grad).max() < 1e-12


def test_fp4_oracle_rounds_to_the_nearest_code():
    """Brute force over the grid and its borders, and the ties by parity."""
    a = np.concatenate([np.linspace(0, 7, 1401), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]])
    got = fp4.nearest(a, fp4.GRID)
    for v, c in zip(a, got):
        d = np.abs(fp4.GRID - v)
        best = np.flatnonzero(d == d.min())
        assert c in best and (len(best) == 1 or c % 2 == 0)
    assert fp4.nearest(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0]), fp4.GRID).tolist() == [0, 2, 2, 4, 4, 6, 6, 7]


def test_fp4_oracle_scales():
    e = fp4.e4m3_values()
    assert e[-1] == 448 and e[1] == 2.0 ** -9 and (np.diff(e) > 0).all()
    W = np.zeros((1, 32), np.float32)
    W[0, 3] = 5.0  # amax in [4, 8): exponent 0
    c, s, v = fp4.quantize(W, "mx")
    assert s.tolist() == [[127]] and v[0, 3] == 4.0 and c[0, 3] == 6
    W[0, 3] = 7.9  # saturates at 6
    assert fp4.quantize(W, "mx")[2][0, 3] == 6.0
    W[0, 3] = 6 * 448 * 4.0
    assert fp4.tensor_scale(W) == 4.0
    assert fp4.tensor_scale(np.nextafter(W, np.inf, dtype=np.float32)) == 8.0
    assert fp4.tensor_scale(np.zeros((1, 32))) == np.float32(2.0 ** -100)
    c, s, v = fp4.quantize(W, "nv", 4.0)
    assert s[0, 0] == 0x7E and s[0, 1] == 0 and v[0, 3] == W[0, 3]


# ------------------------------------------------------------------ refusals of the C ABI


def logprobs(lib, x=FAKE, dt=1, ld=40, T=3, V=40, targets=FAKE, tau=1.0, k=2, lp=FAKE, ent=FAKE, ids=FAKE, top=FAKE):
    return lib.eqat_token_logprobs(P(x), dt, ld, T, V, P(targets), tau, k, P(lp), P(ent), P(ids), P(top), None)


def test_token_logprobs_refusals(lib):
    assert logprobs(lib, dt=2) == DTYPE
    assert logprobs(lib, T=-1) == SHAPE
    assert logprobs(lib, V=0) == SHAPE
    assert logprobs(lib, ld=39) == SHAPE
    assert logprobs(lib, V=(1 << 30) + 1, ld=(1 << 30) + 1) == SHAPE
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-7, 1e7):
        assert logprobs(lib, tau=tau) == UNSUP
    assert logprobs(lib, k=-1) == UNSUP and logprobs(lib, k=129) == UNSUP
    assert logprobs(lib, x=0) == NULL and logprobs(lib, targets=0) == NULL
    assert logprobs(lib, ids=0) == NULL and logprobs(lib, top=0) == NULL
    assert logprobs(lib, x=FAKE + 8) == ALIGN
    assert logprobs(lib, targets=FAKE + 4) == ALIGN
    assert logprobs(lib, lp=FAKE + 2) == ALIGN
    assert logprobs(lib, T=0, x=0, targets=0, lp=0, ent=0, ids=0, top=0) == OK


def distill(lib, x=FAKE, dt=1, ld=40, T=3, V=40, ids=FAKE, tlp=FAKE, k=4, tau=1.0, flags=0, w=FAKE, loss=FAKE, dx=FAKE):
    return lib.eqat_distill_topk(P(x), dt, ld, T, V, P(ids), P(tlp), k, tau, flags, P(w), P(loss), P(dx), None)


def test_distill_refusals(lib):
    assert distill(lib, dt=2) == DTYPE
    assert distill(lib, ld=30) == SHAPE
    assert distill(lib, V=(1 << 19) + 1, ld=(1 << 19) + 1) == SHAPE
    assert distill(lib, k=0) == UNSUP and distill(lib, k=129) == UNSUP
    assert distill(lib, flags=2) == UNSUP
    assert distill(lib, tau=0.0) == UNSUP
    assert distill(lib, ids=0) == NULL and distill(lib, tlp=0) == NULL and distill(lib, x=0) == NULL
    assert distill(lib, dx=FAKE + 2) == ALIGN and distill(lib, ids=FAKE + 4) == ALIGN
    assert distill(lib, loss=0, dx=0) == OK  # nothing asked for
    assert distill(lib, T=0) == OK


def test_distill_gradient_strides(lib):
    """dx has a row stride of its own, which agrees with x's modulo 16 bytes, and does not
    overlap x unless it is x."""
    def call(x=FAKE, dx=FAKE + (1 << 20), ld=40, ld_dx=40, T=3, V=33, dt=1, loss=0, ids=FAKE):
        return lib.eqat_distill_topk_strided(P(x), dt, ld, T, V, P(ids), P(FAKE), 4, 1.0, 0, None, P(loss), P(dx), ld_dx, None)

    # all of these fail at dx, the others below only for want of a device
    assert call(ld_dx=32) == SHAPE and call(ld_dx=1 << 31) == SHAPE
    assert call(ld_dx=41) == SHAPE and call(ld_dx=44) == SHAPE and call(ld_dx=42, dt=0) == SHAPE
    assert call(dx=FAKE + 16) == UNSUP                        # a few entries on
    assert call(dx=FAKE + 80) == UNSUP                        # a row on
    assert call(dx=FAKE, ld_dx=48) == SHAPE                   # x with another stride
    assert call(dx=FAKE + 2 * 40, ld=80, ld_dx=80, V=41) == UNSUP  # side by side, but not quite
    assert call(x=FAKE + 2 * 40, dx=FAKE, ld=80, ld_dx=80, V=41) == UNSUP
    good = [dict(ld_dx=48), dict(ld_dx=44, dt=0), dict(ld_dx=41, T=1), dict(dx=FAKE), dict(dx=FAKE, ld_dx=48, T=1),
            dict(dx=FAKE + 2 * 40, ld=80, ld_dx=80), dict(x=FAKE + 2 * 40, dx=FAKE, ld=80, ld_dx=80),
            dict(dx=FAKE + 3 * 80)]
    if not torch.cuda.is_available():  # (they would run)
        for kw in good:
            assert call(**kw) not in (OK, SHAPE, UNSUP, ALIGN, NULL), kw
    assert call(T=0) == OK and call(dx=0, ld_dx=0) == OK


def test_fp4_refusals(lib):
    st = None
    pack = lambda x=FAKE, dt=1, N=3, K=64, fmt=1, g=FAKE, c=FAKE, s=FAKE: lib.eqat_pack_fp4(  # noqa: E731
        P(x), dt, N, K, fmt, P(g), P(c), P(s), st)
    assert pack(dt=2) == DTYPE
    assert pack(fmt=2) == UNSUP and pack(fmt=0) == UNSUP  # mx has no tensor scale
    assert pack(K=48) == SHAPE and pack(N=-1) == SHAPE
    assert pack(x=0) == NULL and pack(c=0) == NULL and pack(s=0) == NULL
    assert pack(x=FAKE + 8) == ALIGN and pack(g=FAKE + 2) == ALIGN
    assert pack(N=0) == OK
    assert lib.eqat_fake_quant_fp4(P(FAKE), 1, 3, 64, 1, P(FAKE), P(0), st) == NULL
    assert lib.eqat_dequant_fp4(P(FAKE), P(FAKE), 3, 64, 1, P(FAKE), P(FAKE), 2, st) == DTYPE
    assert lib.eqat_fp4_tensor_scale(P(FAKE), 1, 33, P(FAKE), st) == SHAPE
    assert lib.eqat_fp4_tensor_scale(P(FAKE), 1, 32, P(0), st) == NULL
    fwd = lambda X=FAKE, N=16, K=64, fmt=0, g=0, ws=FAKE, n=1 << 20, M=17: lib.eqat_fp4_linear_fwd(  # noqa: E731
        P(X), P(FAKE), P(FAKE), fmt, P(g), P(g), P(FAKE), M, N, K, P(ws), n, st)
    assert fwd(N=12) == SHAPE and fwd(K=40) == SHAPE and fwd(fmt=3) == UNSUP and fwd(g=FAKE) == UNSUP
    assert fwd(ws=0) == WS and fwd(n=100) == WS and fwd(ws=FAKE + 16) == ALIGN
    assert fwd(X=0) == NULL and fwd(M=0) == OK and fwd(N=0) == OK
    bwd = lambda dY=FAKE, dX=FAKE, dW=FAKE, ws=FAKE, n=1 << 20: lib.eqat_fp4_linear_bwd(  # noqa: E731
        P(FAKE), P(FAKE), P(FAKE), 0, P(0), P(0), P(dY), P(dX), P(dW), 3, 16, 64, P(ws), n, st)
    assert bwd(dY=0) == NULL and bwd(dX=FAKE + 2) == ALIGN and bwd(n=8) == WS and bwd(dX=0, dW=0) == OK
    assert lib.eqat_fp4_scale_bytes(129, 96, 1) == 2 * 2 * 512  # 6 blocks of 16: two tiles along K
    assert lib.eqat_fp4_scale_bytes(128, 96, 0) == 512 and lib.eqat_fp4_scale_bytes(1, 20, 0) == 0
    assert lib.eqat_fp4_workspace_bytes(3, 16, 64, 0, 0) == 0  # packed inside the product
    assert lib.eqat_fp4_workspace_bytes(17, 16, 64, 0, 0) == 768 + 512
    assert lib.eqat_fp4_workspace_bytes(3, 16, 64, 0, 1) == 16 * 64 * 2 + 512


def test_fp4_backward_workspace_of_one_gradient(lib):
    """Only the values that a gradient takes have to fit."""
    M, N, K = 300, 24, 64
    w, x = N * K * 2, M * K * 2
    q = lambda b: lib.eqat_fp4_workspace_bytes(M, N, K, 1, b)  # noqa: E731
    assert (q(1), q(2), q(3)) == (w + x, w, x)
    bwd = lambda dX, dW, n: lib.eqat_fp4_linear_bwd(  # noqa: E731
        P(FAKE), P(FAKE), P(FAKE), 1, P(0), P(0), P(FAKE), P(dX), P(dW), M, N, K, P(FAKE), n, None)
    assert bwd(FAKE, 0, w - 1) == WS and bwd(0, FAKE, x - 1) == WS and bwd(FAKE, FAKE, w + x - 1) == WS
    if not torch.cuda.is_available():  # (they would run)
        assert WS not in (bwd(FAKE, 0, w), bwd(0, FAKE, x), bwd(FAKE, FAKE, w + x))


def test_binding_refuses_what_is_no_tensor():
    x, t = torch.zeros(3, 40), torch.zeros(3, dtype=torch.int64)
    tlp = torch.zeros(3, 2)
    W, c = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8)
    s = torch.zeros(1, 1, 512, dtype=torch.uint8)
    for call in [
        lambda: eqat.token_logprobs(None, t),
        lambda: eqat.token_logprobs([[0.0]], t),
        lambda: eqat.distill_topk_fwd(None, t, tlp),
        lambda: eqat.fp4_tensor_scale(None),
        lambda: eqat.pack_fp4(None, "mx"),
        lambda: eqat.fake_quant_fp4(W.tolist(), "mx"),
        lambda: eqat.dequant_fp4(None, s, "mx"),
        lambda: eqat.fp4_linear_fwd(None, c, s, "mx"),
        lambda: eqat.fp4_linear_fwd(W, None, s, "mx"),
        lambda: eqat.fp4_linear_bwd(W, c.tolist(), s, W, "mx"),
    ]:
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        eqat.fp4_scale_shape(8, 64, "fp8")


def test_binding_refusals():
    x, t = torch.zeros(3, 40), torch.zeros(3, dtype=torch.int64)
    ids, tlp = torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2)
    W, c = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8)
    s = torch.zeros(1, 1, 512, dtype=torch.uint8)
    for call in [
        lambda: eqat.token_logprobs(x, t),                       # CPU tensors
        lambda: eqat.token_logprobs(x, t[:2]),
        lambda: eqat.token_logprobs(x[0], t),
        lambda: eqat.token_logprobs(x.t(), torch.zeros(40, dtype=torch.int64)),
        lambda: eqat.token_logprobs(x[:1].expand(3, 40), t),     # overlapping rows
        lambda: eqat.distill_topk_fwd(x, ids, tlp[:, :1]),
        lambda: eqat.distill_topk_bwd(x, ids, tlp, torch.zeros(2)),
        lambda: eqat.distill_topk_step(x, ids, tlp, dlogits=torch.zeros(3, 39)),
        lambda: eqat.pack_fp4(W, "fp8"),
        lambda: eqat.pack_fp4(torch.zeros(8, 40), "mx"),
        lambda: eqat.pack_fp4(W, "nv", codes=c[:, :8]),
        lambda: eqat.pack_fp4(W, "nv", tscale=torch.zeros(2)),
        lambda: eqat.dequant_fp4(c, s[:, :, :8], "mx"),
        lambda: eqat.fp4_linear_fwd(W, c[:, :16], s, "mx"),
        lambda: eqat.fp4_linear_fwd(W, c, s, "mx", Y=torch.zeros(8, 16, dtype=torch.bfloat16)),
        lambda: eqat.fp4_linear_bwd(W, c, s, W, "mx"),
    ]:
        with pytest.raises(ValueError):
            call()
