"""GPU parity of the microscaled 4-bit float operators against the CPU oracle.

Codes, scale bytes, tensor scales and values must match exactly.  Products: with u = 2^-8
the rounding of a bf16 result, and each of the K / 64 block products added to an fp32 sum
within 2^-22 of the sum of magnitudes, |Y - ref| <= u |ref| + (K / 64 + 8) 2^-22
sum |x w|; the backward's plain bf16 products likewise, with steps of 16."""
import numpy as np
import pytest
import torch

import weight_quantization_aware_b200 as eqat
from oracle import fp4 as orc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_quantization_aware_b200 import build
    build.build()
    eqat.load_library()
    assert torch.cuda.is_available()
    yield
    assert eqat.device_error() == 0


def draw(N, K, dtype, seed, sigma=0.02):
    rng = np.random.default_rng(seed)
    w = rng.normal(size=(N, K)).astype(np.float32) * np.float32(sigma)
    w[rng.random((N, K)) < 1e-2] *= 10
    return torch.from_numpy(w).to(dtype)


def f32(t):
    return t.detach().cpu().float().numpy()


def edge_values(N, K, dtype, seed):
    """Values on and next to the borders between codes, zeros, blocks of one value, tiny
    and huge blocks."""
    rng = np.random.default_rng(seed)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, 0.0], np.float32)
    w = rng.choice(mids, (N, K)) * rng.choice([-1.0, 1.0], (N, K))
    w = (w * 2.0 ** rng.integers(-8, 5, (N, 1))).astype(np.float32)
    w *= rng.choice(np.array([1, 1, 1, 1 + 2.0 ** -7, 1 - 2.0 ** -8, 1 + 2.0 ** -23, 1 - 2.0 ** -24], np.float32), (N, K))
    if N > 4:
        w[0] = 0.0
        w[1, : K // 2] = -0.0
        w[2] *= np.float32(2.0 ** -120)
        w[3] *= np.float32(2.0 ** 100)
        w[4, ::16] = 1e-40
    return torch.from_numpy(w.astype(np.float32)).to(dtype)


def check_pack(W, fmt, g):
    N, K = W.shape
    Wd = W.cuda()
    gd = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
    codes, scales = eqat.pack_fp4(Wd, fmt, tscale=gd)
    c, s, v = orc.quantize(f32(W), fmt, g)
    assert np.array_equal(codes.cpu().numpy(), orc.pack(c)), "codes"
    assert np.array_equal(scales.cpu().numpy(), orc.tiles(s)), "scales"
    want = torch.from_numpy(v.astype(np.float32)).to(W.dtype)
    for got in (eqat.fake_quant_fp4(Wd, fmt, tscale=gd), eqat.dequant_fp4(codes, scales, fmt, tscale=gd, dtype=W.dtype)):
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0)), "values"
    return codes, scales, v


SHAPES = [(1, 32), (3, 64), (8, 96), (128, 128), (129, 160), (301, 512), (40, 1056), (257, 4096)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_pack_matches_the_oracle(shape, dtype, fmt):
    W = draw(*shape, dtype, sum(shape))
    g = None
    if fmt == "nv":
        g = float(eqat.fp4_tensor_scale(W.cuda()).item())
        assert np.float32(g) == orc.tensor_scale(f32(W))
    check_pack(W, fmt, g)
    check_pack(edge_values(*shape, dtype, 1), fmt, None if fmt == "mx" else 2.0 ** -4)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_fake_quant_in_place(fmt):
    for dtype in (torch.bfloat16, torch.float32):
        W = draw(1500, 2080, dtype, 4).cuda()
        want = eqat.fake_quant_fp4(W, fmt)
        assert eqat.fake_quant_fp4(W, fmt, W_hat=W) is W and torch.equal(W, want)


@pytest.mark.parametrize("M", [2, 40, 150])
def test_largest_tensor_scales(M):
    """Tensor scales whose product is beyond fp32: a sum of 0 stays 0."""
    g = torch.full((1,), 2.0 ** 100, device="cuda")
    X, W = torch.zeros(M, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(136, 256, dtype=torch.bfloat16, device="cuda")
    X[:, :16], W[:, 16:32] = 2.0 ** 100, 2.0 ** 100
    X[0, 40], W[3, 40] = 2.0 ** 100, -2.0 ** 100
    codes, scales = eqat.pack_fp4(W, "nv", tscale=g)
    Y = f32(eqat.fp4_linear_fwd(X, codes, scales, "nv", tscale=g, x_tscale=g))
    want = np.zeros((M, 136), np.float32)
    want[0, 3] = -np.inf
    assert np.array_equal(Y, want)


@pytest.mark.parametrize("M", [2, 13, 40, 150])
@pytest.mark.parametrize("ex", [100, -100])
def test_tensor_scales_of_opposite_sizes(M, ex):
    """2^100 on one side and 2^-100 on the other: sums near 2^30 and 2 stay what they are,
    whichever scale comes first."""
    K = 256
    gx, gw = (torch.full((1,), 2.0 ** e, device="cuda") for e in (ex, -ex))
    X = torch.full((M, K), 2688.0 * 2.0 ** ex, dtype=torch.bfloat16, device="cuda")
    W = torch.full((136, K), 2688.0 * 2.0 ** -ex, dtype=torch.bfloat16, device="cuda")
    X[1], W[5] = 6 * 2.0 ** (ex - 6), 6 * 2.0 ** (-ex - 6)  # a block scale of 2^-6 and codes of 6
    codes, scales = eqat.pack_fp4(W, "nv", tscale=gw)
    Y = eqat.fp4_linear_fwd(X, codes, scales, "nv", tscale=gw, x_tscale=gx)
    x, w = torch.full((M, 1), 2688.0, dtype=torch.float64), torch.full((136, 1), 2688.0, dtype=torch.float64)
    x[1], w[5] = 6 / 64, 6 / 64
    assert torch.equal(Y.cpu(), (K * x @ w.t()).to(torch.bfloat16))  # all sums are exact in fp32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_any_tensor_scale(dtype):
    """A tensor scale that is not a power of two: the same fp32 operations in the same order."""
    for g in (0.0123, 3.7, 1.0, 1e-3):
        W = draw(33, 256, dtype, 5)
        gd = torch.tensor([g], dtype=torch.float32, device="cuda")
        codes, scales = eqat.pack_fp4(W.cuda(), "nv", tscale=gd)
        c, s, v = orc.quantize(f32(W), "nv", np.float32(g))
        assert np.array_equal(codes.cpu().numpy(), orc.pack(c)) and np.array_equal(scales.cpu().numpy(), orc.tiles(s))
        got = f32(eqat.dequant_fp4(codes, scales, "nv", tscale=gd, dtype=dtype)).astype(np.float64)
        u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(got - v) <= np.abs(v) * (u + 2.0 ** -24)).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_blocks_with_nan_or_infinity(fmt):
    W = draw(9, 128, torch.float32, 2)
    W[2, 40] = float("nan")
    W[5, 0] = float("inf")
    W[8, 127] = -float("inf")
    check_pack(W, fmt, 2.0 ** -10 if fmt == "nv" else None)


def test_tensor_scale_edges():
    for v, want in [(0.0, 2.0 ** -100), (2688.0, 1.0), (2688.0 * (1 + 2.0 ** -23), 2.0), (1e-38, 2.0 ** -100),
                    (3e38, None)]:
        W = torch.zeros(2, 64)
        W[1, 5] = -v
        W[0, 0] = float("nan")  # not a value
        W[0, 1] = float("inf")
        got = eqat.fp4_tensor_scale(W.cuda()).item()
        assert got == (want if want is not None else float(orc.tensor_scale(W.numpy())))
    assert eqat.fp4_tensor_scale(torch.zeros(0, 32, device="cuda")).item() == 2.0 ** -100


def packed(W, fmt, g):
    codes, scales = eqat.pack_fp4(W.cuda(), fmt, tscale=g)
    return codes, scales


def scale_of(t, fmt):
    return eqat.fp4_tensor_scale(t.cuda()) if fmt == "nv" else None


def values(t, fmt, g):
    return orc.quantize(f32(t), fmt, None if g is None else np.float32(g.item()))[2]


CASES = [(1, 8, 32), (1, 128, 256), (2, 136, 64), (7, 264, 320), (16, 512, 1024), (17, 128, 96), (33, 392, 4096),
         (128, 264, 6176), (100, 72, 8256), (17, 1032, 8448),
         (64, 72, 2048), (65, 1000, 512), (128, 256, 288), (129, 264, 320), (300, 520, 1184), (257, 8, 4096),
         (515, 768, 2048),
         # few tokens: K split over the ranks of a cluster, ranks with uneven and with no parts, K past what is
         # packed in the product
         (1, 136, 8192), (16, 264, 4096), (3, 72, 2336), (5, 64, 32768), (13, 1032, 1312), (2, 40, 33024)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c)) for c in CASES])
def test_linear_fwd(case, fmt):
    M, N, K = case
    X, W = draw(M, K, torch.bfloat16, 1, 1.0), draw(N, K, torch.bfloat16, 2)
    gx, gw = scale_of(X, fmt), scale_of(W, fmt)
    codes, scales = packed(W, fmt, gw)
    Y = eqat.fp4_linear_fwd(X.cuda(), codes, scales, fmt, tscale=gw, x_tscale=gx)
    xv, wv = values(X, fmt, gx), values(W, fmt, gw)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    bound = 2.0 ** -8 * np.abs(ref) + (K / 64 + 8) * 2.0 ** -22 * mag + 1e-37
    d = np.abs(f32(Y) - ref)
    assert (d <= bound).all(), f"worst {np.max(d / bound):.3f} of the bound"


def check_product(M, N, K, fmt, repeats=1):
    """Every element of Y against the oracle's packed values (their fp64 product is taken
    on the GPU), every time the same bits."""
    X, W = draw(M, K, torch.bfloat16, 1, 1.0), draw(N, K, torch.bfloat16, 2)
    gx, gw = scale_of(X, fmt), scale_of(W, fmt)
    codes, scales = packed(W, fmt, gw)
    X = X.cuda()
    Ys = [eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=gw, x_tscale=gx) for _ in range(repeats)]
    xv, wv = (torch.from_numpy(v).cuda() for v in (values(X, fmt, gx), values(W, fmt, gw)))
    ref, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    bound = 2.0 ** -8 * ref.abs() + (K / 64 + 8) * 2.0 ** -22 * mag + 1e-37
    d = (Ys[0].double() - ref).abs()
    assert bool((d <= bound).all()), f"worst {(d / bound).max().item():.3f} of the bound"
    for Y in Ys[1:]:
        assert torch.equal(Y, Ys[0])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rest", [8, 40, 104, 136, 168, 200, 224])
def test_pair_product_of_ragged_widths(rest, fmt):
    """The last tile along N ends inside: its chunks past Y are not stored, and the next
    chunk's buffer must still be free.  With 31 x 4 and 41 x 4 tiles on 74 pairs that tile is a
    pair's second and third: in either accumulator."""
    for whole in (30, 40):
        check_product(1000, 256 * whole + rest, 96, fmt, repeats=8)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(2060, 5128, 64), (2060, 5128, 256), (2060, 5128, 288), (1300, 8200, 1312),
                                   (150, 40000, 544), (5000, 2056, 32)])
def test_pair_product_of_several_tiles_per_pair(M, N, K, fmt):
    """More than twice as many tiles as pairs: accumulators taken in turn, whose overlapping
    columns are handed over, and scale buffers that go on from tile to tile; contractions
    shorter than the drain of a tile and longer."""
    check_product(M, N, K, fmt, repeats=3)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_packing_of_several_segments_per_warp(dtype, fmt):
    """Four times as many segments as warps, the second of a row ragged: what is fetched
    ahead is the next segment's, in place too."""
    N, K = 20001, 544
    W = draw(N, K, dtype, 11)
    g = None if fmt == "mx" else 2.0 ** -12
    check_pack(W, fmt, g)
    gd = None if g is None else torch.tensor([g], device="cuda")
    Wd = W.cuda()
    want = eqat.fake_quant_fp4(Wd, fmt, tscale=gd)  # just compared with the oracle
    assert eqat.fake_quant_fp4(Wd, fmt, tscale=gd, W_hat=Wd) is Wd and torch.equal(Wd, want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [3, 200])
def test_linear_fwd_keeps_nan_blocks_to_their_rows(M, fmt):
    N, K = 136, 192
    X, W = draw(M, K, torch.bfloat16, 1, 1.0), draw(N, K, torch.bfloat16, 2)
    X[1, 70] = float("nan")
    W[130, 5] = float("inf")
    g = torch.tensor([2.0 ** -8], device="cuda") if fmt == "nv" else None
    codes, scales = packed(W, fmt, g)
    Y = eqat.fp4_linear_fwd(X.cuda(), codes, scales, fmt, tscale=g, x_tscale=g).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[1] = True
    want[:, 130] = True
    assert torch.equal(torch.isnan(Y), want)


BWD = [(1, 8, 32), (5, 136, 96), (130, 264, 320), (300, 128, 1024)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("case", BWD, ids=["x".join(map(str, c)) for c in BWD])
def test_linear_bwd(case, fmt):
    M, N, K = case
    X, W, dY = draw(M, K, torch.bfloat16, 1, 1.0), draw(N, K, torch.bfloat16, 2), draw(M, N, torch.bfloat16, 3, 0.01)
    gx, gw = scale_of(X, fmt), scale_of(W, fmt)
    codes, scales = packed(W, fmt, gw)
    dX, dW = eqat.fp4_linear_bwd(X.cuda(), codes, scales, dY.cuda(), fmt, tscale=gw, x_tscale=gx)
    xv, wv, dy = values(X, fmt, gx), values(W, fmt, gw), f32(dY).astype(np.float64)
    for got, a, b, n in ((dX, dy, wv, N), (dW, dy.T, xv, M)):
        ref, mag = a @ b, np.abs(a) @ np.abs(b)
        bound = 2.0 ** -8 * np.abs(ref) + (n / 16 + 8) * 2.0 ** -22 * mag + 1e-37
        d = np.abs(f32(got) - ref)
        assert (d <= bound).all(), f"worst {np.max(d / bound):.3f} of the bound"
    only, none = eqat.fp4_linear_bwd(X.cuda(), codes, scales, dY.cuda(), fmt, tscale=gw, x_tscale=gx, need_dw=False)
    assert none is None and torch.equal(only, dX)


@pytest.mark.parametrize("M,N,K", [(4100, 264, 2080), (264, 8200, 2080), (3000, 3000, 544), (2060, 136, 8224), (70, 5128, 4128)])
def test_backward_of_uneven_contractions(M, N, K):
    """Both contractions in one launch, one of them several times as deep as the other (their
    tiles are dealt by cost), or with several tiles per pair; ragged in every size."""
    fmt = "nv"
    X, W, dY = draw(M, K, torch.bfloat16, 1, 1.0), draw(N, K, torch.bfloat16, 2), draw(M, N, torch.bfloat16, 3, 0.01).cuda()
    gx, gw = scale_of(X, fmt), scale_of(W, fmt)
    codes, scales = packed(W, fmt, gw)
    X = X.cuda()
    dX, dW = eqat.fp4_linear_bwd(X, codes, scales, dY, fmt, tscale=gw, x_tscale=gx)
    xv, wv = (torch.from_numpy(values(t, fmt, g)).cuda() for t, g in ((X, gx), (W, gw)))
    dy = dY.double()
    for got, a, b, n in ((dX, dy, wv, N), (dW, dy.t(), xv, M)):
        ref, mag = a @ b, a.abs() @ b.abs()
        bound = 2.0 ** -8 * ref.abs() + (n / 16 + 8) * 2.0 ** -22 * mag + 1e-37
        assert bool(((got.double() - ref).abs() <= bound).all())
    again = eqat.fp4_linear_bwd(X, codes, scales, dY, fmt, tscale=gw, x_tscale=gx)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


@pytest.mark.parametrize("M", [3, 16, 40, 128, 300])
def test_product_with_any_tensor_scale(M):
    """Tensor scales that are no power of two (amax / 2688, as other packers write): the
    forward multiplies exact codes and scales, and the fp32 sum by both tensor scales (two
    roundings; the oracle rounds each block's scale times g, two more: 4 2^-24 in all).  The
    backward's values are those rounded to bf16."""
    N, K = 264, 1184
    X, W, dY = draw(M, K, torch.bfloat16, 1, 1.0), draw(N, K, torch.bfloat16, 2), draw(M, N, torch.bfloat16, 3, 0.01)
    gx, gw = ((t.float().abs().max() / 2688).reshape(1).cuda() for t in (X, W))
    codes, scales = packed(W, "nv", gw)
    Y = eqat.fp4_linear_fwd(X.cuda(), codes, scales, "nv", tscale=gw, x_tscale=gx)
    xv, wv = values(X, "nv", gx), values(W, "nv", gw)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    bound = 2.0 ** -8 * np.abs(ref) + (K / 64 + 9) * 2.0 ** -22 * mag
    assert (np.abs(f32(Y) - ref) <= bound).all()
    dX, dW = eqat.fp4_linear_bwd(X.cuda(), codes, scales, dY.cuda(), "nv", tscale=gw, x_tscale=gx)
    xb, wb = (f32(torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)).astype(np.float64) for v in (xv, wv))
    assert not np.array_equal(xb, xv) and (np.abs(wb - wv) <= 2.0 ** -8 * np.abs(wv)).all()
    dy = f32(dY).astype(np.float64)
    for got, a, b, n in ((dX, dy, wb, N), (dW, dy.T, xb, M)):
        ref, mag = a @ b, np.abs(a) @ np.abs(b)
        bound = 2.0 ** -8 * np.abs(ref) + (n / 16 + 8) * 2.0 ** -22 * mag + 1e-37
        assert (np.abs(f32(got) - ref) <= bound).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_backward_of_one_gradient(fmt):
    """Each gradient alone, in a workspace of its own size and no byte more: the same bits as
    together, and nothing written past the workspace."""
    M, N, K = 301, 136, 544
    X, W, dY = (draw(*s, torch.bfloat16, i, 1.0) for i, s in enumerate([(M, K), (N, K), (M, N)]))
    X, dY = X.cuda(), dY.cuda()
    g = scale_of(W, fmt)
    codes, scales = packed(W, fmt, g)
    want = eqat.fp4_linear_bwd(X, codes, scales, dY, fmt, tscale=g)
    for dx, dw in ((True, False), (False, True), (True, True)):
        n = eqat.fp4_workspace(M, N, K, fmt, backward=True, need_dx=dx, need_dw=dw).numel()
        buf = torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda")
        for ws in (None, buf[:n]):
            got = eqat.fp4_linear_bwd(X, codes, scales, dY, fmt, tscale=g, need_dx=dx, need_dw=dw, ws=ws)
            for a, b, need in zip(got, want, (dx, dw)):
                assert torch.equal(a, b) if need else a is None
        assert bool((buf[n:] == 7).all())
        with pytest.raises(eqat.EqatError):
            eqat.fp4_linear_bwd(X, codes, scales, dY, fmt, tscale=g, need_dx=dx, need_dw=dw, ws=buf[:n - 1])
    assert eqat.fp4_linear_bwd(X, codes, scales, dY, fmt, tscale=g, need_dx=False, need_dw=False) == (None, None)


def test_backward_matches_differences():
    """The product is linear in each packed operand: dX against the change of sum(dY Y)
    when a block of X moves along the packed grid by whole codes (both exact)."""
    M, N, K, fmt = 4, 64, 64, "mx"
    X = torch.full((M, K), 1.0, dtype=torch.bfloat16)
    X[:, ::32] = 4.0  # every block's scale stays 1
    W, dY = draw(N, K, torch.bfloat16, 4), draw(M, N, torch.bfloat16, 5)
    codes, scales = packed(W, fmt, None)
    dX, _ = eqat.fp4_linear_bwd(X.cuda(), codes, scales, dY.cuda(), fmt)
    up, dn = X.clone(), X.clone()
    up[2, 7], dn[2, 7] = 1.5, 0.5
    wv = values(W, fmt, None)
    dy = f32(dY).astype(np.float64)
    num = (dy * (values(up, fmt, None) @ wv.T - values(dn, fmt, None) @ wv.T)).sum()
    assert abs(num - float(dX[2, 7])) <= 2.0 ** -7 * abs(num) + 1e-6 * np.abs(dy[2]) @ np.abs(wv[:, 7])


def test_workspaces_outputs_and_empty_calls():
    M, N, K, fmt = 20, 64, 128, "nv"
    X, W = draw(M, K, torch.bfloat16, 1, 1.0).cuda(), draw(N, K, torch.bfloat16, 2)
    g = scale_of(W, fmt)
    codes, scales = packed(W, fmt, g)
    want = eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=g)
    assert eqat.fp4_workspace(16, N, K, fmt).numel() == 1  # nothing needed
    ws = eqat.fp4_workspace(M, N, K, fmt).fill_(255)
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=g, ws=ws, Y=Y)
    assert got.data_ptr() == Y.data_ptr() and torch.equal(got, want)
    with pytest.raises(eqat.EqatError):
        eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=g, ws=ws[:256])
    assert eqat.fp4_linear_fwd(X[:0], codes, scales, fmt).shape == (0, N)
    dX, dW = eqat.fp4_linear_bwd(X[:0], codes, scales, torch.empty(0, N, dtype=torch.bfloat16, device="cuda"), fmt)
    assert dX.shape == (0, K) and dW.shape == (N, K) and not dW.any()
    with pytest.raises(eqat.EqatError):
        eqat.fp4_linear_fwd(X, codes, eqat.pack_fp4(W.cuda(), "mx")[1], "mx", tscale=g)


def test_graph_and_side_stream():
    M, N, K, fmt = 9, 264, 512, "nv"
    X, W = draw(M, K, torch.bfloat16, 1, 1.0).cuda(), draw(N, K, torch.bfloat16, 2).cuda()
    g = eqat.fp4_tensor_scale(W)
    codes, scales = eqat.pack_fp4(W, fmt, tscale=g)
    want = eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=g)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2 = eqat.fp4_tensor_scale(W)
        c2, s2 = eqat.pack_fp4(W, fmt, tscale=g2)
        Y = eqat.fp4_linear_fwd(X, c2, s2, fmt, tscale=g2)
    X.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=g))


def test_a_distillation_step_through_a_packed_output_layer():
    """Teacher's logits -> alternatives -> the loss of a packed student -> its gradients,
    against the same chain in fp64 with the kernels' packed values and bf16 logits."""
    from oracle import rows
    M, V, K, k, fmt = 70, 1024, 256, 16, "nv"
    X, W = draw(M, K, torch.bfloat16, 1, 1.0).cuda(), draw(V, K, torch.bfloat16, 2, 0.1)
    T = (X.float() @ W.cuda().float().t()).to(torch.bfloat16)
    lp, ent, ids, tlp = eqat.token_logprobs(T, torch.arange(M, device="cuda"), top_k=k)
    gw, gx = eqat.fp4_tensor_scale(W.cuda()), eqat.fp4_tensor_scale(X)
    codes, scales = eqat.pack_fp4(W.cuda(), fmt, tscale=gw)
    Y = eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=gw, x_tscale=gx)
    w = torch.full((M,), 1.0 / M, device="cuda")
    loss, dY = eqat.distill_topk_step(Y, ids, tlp, weight=w, tail=True)
    dX, dW = eqat.fp4_linear_bwd(X, codes, scales, dY, fmt, tscale=gw, x_tscale=gx)
    want_l, want_g = rows.distill_topk(f32(Y), ids.cpu().numpy(), f32(tlp), f32(w), 1.0, True)
    assert np.allclose(f32(loss), want_l, rtol=1e-4, atol=1e-7)
    xv, wv, dy = values(X, fmt, gx), values(W, fmt, gw), f32(dY).astype(np.float64)
    assert np.abs(dy - want_g).max() <= 2.0 ** -8 * np.abs(want_g).max() + 1e-9
    for got, a, b, n in ((dX, dy, wv, V), (dW, dy.T, xv, M)):
        ref, mag = a @ b, np.abs(a) @ np.abs(b)
        assert (np.abs(f32(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (n / 16 + 8) * 2.0 ** -22 * mag).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_matrices_past_32_bit_offsets(fmt):
    """More than 2^31 values: the last rows are what packing and multiplying them alone gives."""
    N, K = 65544, 32768
    W = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    W[: N - 8] = 0.25
    W[N - 8:] = draw(8, K, torch.bfloat16, 5).cuda()
    tail = W[N - 8:].clone()
    g = None
    if fmt == "nv":
        g = eqat.fp4_tensor_scale(W)
        assert torch.equal(g, eqat.fp4_tensor_scale(torch.cat([tail, W[:1]])))
    codes, scales = eqat.pack_fp4(W, fmt, tscale=g)
    want = eqat.fake_quant_fp4(tail, fmt, tscale=g)
    assert torch.equal(eqat.fake_quant_fp4(W, fmt, tscale=g, W_hat=W)[N - 8:], want)
    assert torch.equal(W[N - 9], eqat.fake_quant_fp4(torch.full((1, K), 0.25, dtype=torch.bfloat16, device="cuda"), fmt,
                                                     tscale=g)[0])
    W.zero_()
    assert torch.equal(eqat.dequant_fp4(codes, scales, fmt, tscale=g, out=W)[N - 8:], want)
    del W
    wv = f32(want).astype(np.float64)
    for M in (3, 40, 130):
        X = draw(M, K, torch.bfloat16, M, 1.0)
        gx = scale_of(X, fmt)
        Y = eqat.fp4_linear_fwd(X.cuda(), codes, scales, fmt, tscale=g, x_tscale=gx)
        xv = values(X, fmt, gx)
        ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        bound = 2.0 ** -8 * np.abs(ref) + (K / 64 + 8) * 2.0 ** -22 * mag + 1e-37
        assert (np.abs(f32(Y[:, N - 8:]) - ref) <= bound).all()
        assert torch.equal(Y[:, 0], Y[:, N - 9])  # equal rows of W, the first and the last of them


def test_calls_at_once_on_three_streams():
    """Products of a few, some and many tokens and a distillation step, in flight together
    on streams of their own: the same bits as alone."""
    from weight_quantization_aware_b200 import distill_topk_step
    W = draw(2056, 4096, torch.bfloat16, 6).cuda()
    calls = []
    for fmt, M in (("nv", 4), ("mx", 40), ("nv", 300)):
        g = scale_of(W, fmt)
        codes, scales = eqat.pack_fp4(W, fmt, tscale=g)
        X = draw(M, 4096, torch.bfloat16, M, 1.0).cuda()
        calls.append(lambda X=X, c=codes, s=scales, f=fmt, g=g: eqat.fp4_linear_fwd(X, c, s, f, tscale=g, x_tscale=g))
    z = draw(500, 3001, torch.bfloat16, 7, 2.0).cuda()
    ids = torch.arange(20, device="cuda").repeat(500, 1)
    tlp = torch.full((500, 20), -4.0, device="cuda")
    calls.append(lambda: distill_topk_step(z, ids, tlp, tail=True)[1])
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(60):
        with torch.cuda.stream(streams[i % 3]):
            j = (i // 2) % len(calls)
            got.append((j, calls[j]()))
    torch.cuda.synchronize()
    for j, t in got:
        assert torch.equal(t, want[j])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(17, 8, 32), (40, 136, 32), (64, 8, 96), (100, 1000, 32), (128, 8, 4064), (129, 8, 32)])
def test_products_of_short_sides(M, N, K, fmt):
    check_product(M, N, K, fmt, repeats=2)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_product_past_32_bit_offsets_of_y(fmt):
    """More than 2^31 products: the last rows and columns are what their operands give alone
    (one stage of K, the same sums in either call), and the backward of the last rows."""
    M, N, K = 40968, 60008, 64
    X, W = draw(M, K, torch.bfloat16, 1, 1.0).cuda(), draw(N, K, torch.bfloat16, 2).cuda()
    gx, gw = scale_of(X, fmt), scale_of(W, fmt)
    codes, scales = eqat.pack_fp4(W, fmt, tscale=gw)
    Y = eqat.fp4_linear_fwd(X, codes, scales, fmt, tscale=gw, x_tscale=gx)
    assert Y.numel() > 1 << 31
    want = eqat.fp4_linear_fwd(X[-300:], codes, scales, fmt, tscale=gw, x_tscale=gx)
    assert torch.equal(Y[-300:], want)
    c, s = eqat.pack_fp4(W[-264:], fmt, tscale=gw)
    assert torch.equal(Y[:, -264:], eqat.fp4_linear_fwd(X, c, s, fmt, tscale=gw, x_tscale=gx))
    dX, _ = eqat.fp4_linear_bwd(X, codes, scales, Y, fmt, tscale=gw, x_tscale=gx, need_dw=False)
    dy, wv = Y[-300:].double(), torch.from_numpy(values(W, fmt, gw)).cuda()
    ref, mag = dy @ wv, dy.abs() @ wv.abs()
    bound = 2.0 ** -8 * ref.abs() + (N / 16 + 8) * 2.0 ** -22 * mag
    assert bool(((dX[-300:].double() - ref).abs() <= bound).all())


def test_first_calls_inside_a_capture():
    """A process whose very first calls are captured: nothing of a kernel's preparation may
    need the stream."""
    import subprocess
    import sys
    code = """
import torch, weight_quantization_aware_b200 as eqat
x = torch.randn(300, 1000, device="cuda", dtype=torch.bfloat16)
X, W = x[:40, :64].contiguous(), x[:264, :64].contiguous()
XL = x[:, :64].contiguous()
t = torch.arange(300, device="cuda")
def run():
    out = list(eqat.token_logprobs(x, t, top_k=5))
    out += eqat.distill_topk_step(x, out[2], out[3], tail=True)
    g = eqat.fp4_tensor_scale(W)
    c, s = eqat.pack_fp4(W, "nv", tscale=g)
    for a in (X[:2], X, XL):
        y = eqat.fp4_linear_fwd(a, c, s, "nv", tscale=g)
        out += [y, *eqat.fp4_linear_bwd(a, c, s, y, "nv", tscale=g)]
    return out
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, run()):
    assert torch.equal(a, b)
assert eqat.device_error() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
