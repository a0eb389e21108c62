"""GPU parity of token_logprobs and distill_topk_* against the fp64 oracle.

Tolerances, derived once.  A thread adds about V / 512 terms of one sign into each of two
fp32 sums and the block joins 512 of them in 13 steps, so S has a relative error of at
most (V / 512 + 16) 2^-24 from the additions; each term 2^y carries 2^-22 from ex2 and,
from two roundings of y, |y| 2^-23 ln 2, which weighted by 2^y stays below 2^-23.  So
ln S is within tol(V) = (V / 512 + 32) 2^-24 + 2^-21, absolutely.  Values that are
rounded to fp32 at the end add 2^-24 of themselves.  (On short rows, V <= 16384, a thread
of the narrow block adds up to V / 128 terms: of either sign and half an ulp of a growing
sum at most, 128 roundings stay within 16 2^-24 at four standard deviations.)
"""
import numpy as np
import pytest
import torch

import weight_quantization_aware_b200 as eqat
from oracle import rows as orc

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_quantization_aware_b200 import build
    build.build()
    eqat.load_library()
    assert torch.cuda.is_available()
    yield
    assert eqat.device_error() == 0


def tol(V):
    return (V / 512 + 32) * 2.0 ** -24 + 2.0 ** -21


def make(T, V, dtype, seed, ld=None):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, V)) * 3
    x[np.arange(T), rng.integers(0, V, T)] += 8 * rng.random(T)
    t = torch.from_numpy(x).to(dtype)
    if ld is None:
        return t.cuda()
    wide = torch.full((T, ld), float("nan"), dtype=dtype)  # what lies past a row is never read
    wide[:, :V] = t
    return wide.cuda()[:, :V]


def f64(t):
    return t.detach().cpu().double().numpy()


def same(got, want, bound, name):
    """Equal where not finite, within `bound` elsewhere."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True), f"{name}: non-finite values differ"
    d = np.abs(got[fin] - want[fin])
    b = np.broadcast_to(bound, want.shape)[fin]
    assert np.isfinite(got[fin]).all() and (d <= b).all(), f"{name}: worst {np.max(d / b):.3f} of the bound"


def check_logprobs(x, targets, k, tau=1.0):
    lp, ent, ids, top = eqat.token_logprobs(x, targets, top_k=k, temperature=tau)
    V = x.shape[1]
    xn = f64(x)
    w_lp, w_ent, w_ids, w_top = orc.token_logprobs(xn, targets.cpu().numpy(), k, tau)
    e = tol(V)
    same(f64(lp), w_lp, e + np.abs(np.nan_to_num(w_lp, neginf=0)) * 2.0 ** -23, "logprob")
    # H = ln S - ln 2 A / S: A's relative error is S's plus one rounding of each y
    span = np.abs(np.nan_to_num(w_ent)) + np.log(V)  # bounds E|y| ln 2
    same(f64(ent), w_ent, e * (2 + 3 * span), "entropy")
    if k:
        assert np.array_equal(ids.cpu().numpy(), w_ids), "ids"
        same(f64(top), w_top, e + np.abs(np.nan_to_num(w_top, neginf=0)) * 2.0 ** -23, "top")
    else:
        assert ids is None and top is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (1, 2, 0), (3, 7, 7), (2, 33, 128), (5, 1000, 5), (4, 2049, 128),
                                   (9, 32000, 1), (3, 50001, 64), (700, 513, 20), (2, 131075, 100), (150, 66001, 0), (20, 70003, 0),
                                   (1300, 301, 32), (1300, 301, 33), (1300, 77, 128), (500, 3001, 7), (500, 8001, 0),
                                   (2500, 40, 40)])
def test_logprobs(T, V, k, dtype):
    x = make(T, V, dtype, T * V)
    g = torch.Generator().manual_seed(3)
    check_logprobs(x, torch.randint(0, V, (T,), generator=g).cuda(), min(k, 128))


def test_logits_beyond_two_to_the_31():
    """m c = RN(m c) + up to 128: 2^-y and 2^y of that leave fp32 on either side.  Entries
    are at least 128 apart there, so that a row's probability is that of its largest."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = 1.5e9 + 1.4e9 * torch.rand(3000, 64, generator=gen, device="cuda")
    x[1::2] *= -1
    check_logprobs(x, x.argmax(1), 3)
    check_logprobs(x, torch.arange(3000, device="cuda") % 64, 0)
    ids = torch.arange(6, device="cuda").repeat(3000, 1)
    tlp = torch.log_softmax(torch.randn(3000, 7, generator=gen, device="cuda"), 1)[:, :6].contiguous()
    for tail in (False, True):
        want_l, want_g = orc.distill_topk(f64(x), ids.cpu().numpy(), f64(tlp), None, 1.0, tail)
        loss, grad = eqat.distill_topk_step(x, ids, tlp, tail=tail)
        # q_i within 2^-21 of itself, z - lse within 2^-53 of z, the loss rounded once
        assert np.abs(f64(loss) - want_l).max() <= 2.0 ** -20 * np.abs(want_l).max()
        assert np.abs(f64(grad) - want_g).max() <= 2.0 ** -20


@pytest.mark.parametrize("tau", [0.25, 3.0, 1e-6, 1e6])
def test_logprobs_temperature(tau):
    x = make(6, 4097, torch.float32, 1)
    t = torch.arange(6, device="cuda")
    lp, ent, _, _ = eqat.token_logprobs(x, t, temperature=tau)
    w_lp, w_ent, _, _ = orc.token_logprobs(f64(x), t.cpu().numpy(), 0, tau)
    # every y is rounded twice: at an extreme temperature the error of the largest
    # scaled logit counts, 2^-23 of it
    big = np.abs(w_lp) * 2.0 ** -22
    same(f64(lp), w_lp, tol(4097) + big, "logprob")
    same(f64(ent), w_ent, tol(4097) * (2 + 3 * (w_ent + np.log(4097))), "entropy")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_logprobs_strides_masks_and_bad_rows(dtype):
    T, V = 12, 3001
    for ld in (3001, 3002, 3008, 4000):
        x = make(T, V, dtype, ld, ld)
        lowest = torch.finfo(dtype).min
        x[1, 5:] = -float("inf")           # five entries left
        x[2] = -float("inf")               # nothing left
        x[3, 100:] = lowest                # masked by the type's lowest value
        x[4] = lowest                      # a whole row of it: uniform
        x[5, 17] = float("nan")
        x[6, 18] = float("inf")
        x[7] = 0.0                         # all equal
        x[8, ::2] = 0.0                    # ties of both zeros
        x[8, 1::2] = -0.0
        x[9, 1:] = -float("inf")           # one entry left
        t = torch.tensor([0, 3, 3, 200, 1, 0, 0, 9, 9, 0, -100, V], device="cuda")
        check_logprobs(x, t, 40)
        check_logprobs(x, torch.full((T,), -1, device="cuda"), 0)


@pytest.mark.parametrize("tau", [1.0, 0.05, 20.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_masks_of_every_size(dtype, tau):
    """Finite masks from -1e4 to the type's lowest value over whole threads' entries, at
    the front, at the back and alternating, rows of one such value, and rows around
    it: the sums must come from the entries that are left."""
    V = 9001
    masks = [-1e4, -1e7, -1e8, -1e10, -1e15, -1e30, torch.finfo(dtype).min, -float("inf")]
    x = make(4 * len(masks), V, dtype, 5)
    for i, m in enumerate(masks):
        x[4 * i, :8500] = m
        x[4 * i + 1, 300:] = m
        x[4 * i + 2, torch.arange(V, device="cuda") % 7 != 3] = m
        x[4 * i + 3] = m
        x[4 * i + 3, ::5] = m * (1.01 if abs(m) < 1e37 else 0.99)
    t = torch.full((len(x),), 8999, device="cuda")
    xn = f64(x)
    with np.errstate(invalid="ignore", over="ignore"):
        zmax = np.where(np.isfinite(xn.max(1)), np.abs(xn.max(1)), 0) / tau
    lp, ent, ids, top = eqat.token_logprobs(x, t, top_k=12, temperature=tau)
    w_lp, w_ent, w_ids, w_top = orc.token_logprobs(xn, t.cpu().numpy(), 12, tau)
    with np.errstate(over="ignore"):  # beyond fp32 a log probability is -inf
        w_lp, w_top = w_lp.astype(np.float32).astype(np.float64), w_top.astype(np.float32).astype(np.float64)
    # y = (x - m) c is rounded to 2^-23 of itself, which in a far row may be large where it counts (|y| < 150)
    e = tol(V) + 2.0 ** -22 * np.minimum(zmax, 100)
    same(f64(lp), w_lp, e + np.abs(np.nan_to_num(w_lp, neginf=0)) * 2.0 ** -22, "logprob")
    same(f64(ent), w_ent, e * (2 + 3 * (np.abs(w_ent) + np.log(V))), "entropy")
    assert np.array_equal(ids.cpu().numpy(), w_ids)
    same(f64(top), w_top, e[:, None] + np.abs(np.nan_to_num(w_top, neginf=0)) * 2.0 ** -22, "top")
    gen = torch.Generator(device="cuda").manual_seed(2)
    tids = torch.stack([torch.randperm(V, generator=gen, device="cuda")[:9] for _ in range(len(x))])
    tlp = torch.log_softmax(torch.randn(len(x), 10, generator=gen, device="cuda"), 1)[:, :9].contiguous()
    for tail in (False, True):
        want_l, want_g = orc.distill_topk(xn, tids.cpu().numpy(), f64(tlp), None, tau, tail)
        loss, grad = eqat.distill_topk_step(x, tids, tlp, temperature=tau, tail=tail)
        with np.errstate(over="ignore"):
            want_l = want_l.astype(np.float32).astype(np.float64)
        same(f64(loss), want_l, 4 * e + np.abs(np.nan_to_num(want_l, posinf=0)) * 2.0 ** -21 + 1e-37, "loss")
        rel = 4 * e[:, None] + 2.0 ** -19 + 150 * 2.0 ** -23
        same(f64(grad), want_g, 3 * rel / tau + np.abs(want_g) * HALF[dtype] + 1e-37, "gradient")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_top_k_of_uneven_and_tied_rows(dtype):
    """Rows whose candidates overflow the selection's buffer: large values in one stride
    of the walk, few distinct values, everything equal but a handful."""
    V = 20011
    x = make(6, V, dtype, 2)
    x[0] = 1.0
    x[1] = (torch.arange(V) % 3).to(dtype)
    x[2] = 1.0
    x[2, torch.tensor([19999, 7, 12345])] = 2.0
    x[2, 20000:] = 0.5
    x[3] = torch.sort(x[3])[0]
    x[4] = torch.round(x[4])
    x[5] = -5.0
    x[5, V - 1] = -4.0
    for k in (1, 3, 64, 128):
        check_logprobs(x, torch.arange(6, device="cuda"), k)
    # the narrow block: short rows, many of them
    y = x[:, :4001].repeat(90, 1).contiguous()
    y[::6, 100:] += 0.0
    for k in (3, 32):
        check_logprobs(y, torch.arange(len(y), device="cuda"), k)


def check_distill(x, ids, tlp, w, tau, tail, least=1e-37):
    V = x.shape[1]
    want_l, want_g = orc.distill_topk(f64(x), ids.cpu().numpy(), f64(tlp), None if w is None else f64(w), tau, tail)
    loss, grad = eqat.distill_topk_step(x, ids, tlp, weight=w, temperature=tau, tail=tail)
    wn = np.ones(x.shape[0]) if w is None else np.abs(f64(w))
    e = 2 * tol(V)  # ln S, and ln of the sum outside the slots
    # the loss multiplies those by masses that add up to 1; the largest |ln p| by 2^-22
    same(f64(loss), want_l, wn * 2 * e + np.abs(np.nan_to_num(want_l, posinf=0)) * 2.0 ** -22 + 1e-37, "loss")
    # a gradient is a difference of masses, each with S's relative error, 2^-21, and
    # |y| 2^-23 of its exponent (|y| <= 150 where 2^y is not 0)
    xz = f64(x) / tau
    with np.errstate(invalid="ignore", over="ignore"):
        z = xz - np.max(np.where(np.isnan(xz), -np.inf, xz), 1, keepdims=True)
        p = np.nan_to_num(np.exp(z) / np.exp(z).sum(1, keepdims=True))
    mag = 2 * p + np.abs(np.nan_to_num(want_g)) / np.maximum(wn[:, None], 1e-30) * tau
    rel = e + 2.0 ** -20 + 150 * 2.0 ** -23
    bound = wn[:, None] / tau * mag * rel + np.abs(np.nan_to_num(want_g)) * (HALF[x.dtype] + 2.0 ** -22) + least
    same(f64(grad), want_g, bound, "gradient")
    # the separate calls give the same bits
    assert torch.equal(eqat.distill_topk_fwd(x, ids, tlp, weight=w, temperature=tau, tail=tail).nan_to_num(7.0), loss.nan_to_num(7.0))
    dl = torch.ones(x.shape[0], device="cuda") if w is None else w
    g2 = eqat.distill_topk_bwd(x, ids, tlp, dl, temperature=tau, tail=tail)
    assert torch.equal(g2.nan_to_num(7.0), grad.nan_to_num(7.0))
    return loss, grad


def teacher(x, k, seed, tau=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    y = x.float() + torch.randn(x.shape, generator=g, device="cuda")
    t = torch.zeros(x.shape[0], dtype=torch.int64, device="cuda")
    _, _, ids, tlp = eqat.token_logprobs(y, t, top_k=k, temperature=tau)
    return ids, tlp


@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,k,tau", [(1, 1, 1, 1.0), (2, 5, 5, 1.0), (3, 9, 4, 2.0), (4, 1000, 1, 0.7),
                                       (700, 515, 16, 1.0), (5, 32000, 128, 2.0), (2, 131075, 32, 1.0),
                                       (150, 66001, 40, 1.0), (20, 70003, 7, 0.5), (2, 300007, 9, 1.0),
                                       (1300, 301, 32, 1.0), (500, 8001, 128, 2.0), (2500, 40, 40, 1.0)])
def test_distill(T, V, k, tau, dtype, tail):
    x = make(T, V, dtype, T + V)
    ids, tlp = teacher(x, k, V, tau)
    w = torch.linspace(0.0, 1.0, T, device="cuda") if T > 1 else None
    check_distill(x, ids, tlp, w, tau, tail)


@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_distill_edges(dtype, tail):
    T, V, k = 14, 2003, 6
    for ld in (2003, 2004, 2048):
        x = make(T, V, dtype, ld, ld)
        clean = make(T, V, dtype, ld)
        ids, tlp = teacher(clean, k, 9)
        inf = float("inf")
        ids[1, 2:] = -1                        # empty slots
        ids[2] = -1                            # a teacher without alternatives
        tlp[3] = -inf                          # alternatives without mass
        x[4] = -inf                            # a student without entries
        x[5, int(ids[5, 1])] = -inf            # a masked entry under a slot with mass
        ids[6, 4] = ids[6, 0]                  # an id given twice, and three times
        ids[7, 1] = ids[7, 2] = ids[7, 5]
        ids[8, 0] = V                          # outside the vocabulary
        x[9, 3] = float("nan")
        x[10, 3] = inf
        tlp[11, 0] = inf
        keep = x[12, ids[12]].clone()          # nothing outside the slots
        x[12] = -inf
        x[12, ids[12]] = keep
        x[13] = torch.finfo(dtype).min         # uniform
        check_distill(x, ids, tlp, None, 1.0, tail)
        w = torch.ones(T, device="cuda")
        w[9] = w[8] = 0.0                      # rows of weight 0 are not looked at
        w[3] = -2.0
        check_distill(x, ids, tlp, w, 1.5, tail)


@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_what_an_empty_slot_holds_is_ignored(dtype, tail):
    inf, V = float("inf"), 2003
    x = make(8, V, dtype, 6)
    ids, tlp = teacher(x, 40, 9)
    for t, v in enumerate([float("nan"), inf, -inf, 0.0, 1e30, 3e38, -3e38, float("nan")]):
        ids[t, [3, 35]] = -1 - t
        tlp[t, [3, 35]] = v
    check_distill(x, ids, tlp, None, 1.0, tail)
    ids[7] = -1
    tlp[7] = float("nan")
    check_distill(x, ids, tlp, None, 1.0, tail)


def test_distill_tail_does_not_cancel():
    """Nearly all mass on the slots: the student's mass outside them is far below 2^-24."""
    V, k = 5000, 3
    x = make(3, V, torch.float32, 4)
    x[:, :k] += 40.0
    ids = torch.arange(k, device="cuda").repeat(3, 1)
    tlp = torch.log(torch.tensor([[0.5, 0.3, 0.1], [0.4, 0.4, 0.2 - 1e-4], [0.2, 0.2, 0.2]], device="cuda"))
    check_distill(x, ids, tlp, None, 1.0, True)


@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_many_rows_give_the_same_bits_every_time(dtype, tail):
    """Several rows per block, whose chunks reuse the ring's slots many times over: every
    run of the step, and the loss alone, agree bit for bit, and sampled rows agree with
    the oracle."""
    T, V, k = 1500, 32000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(T, V, generator=g, device="cuda") * 2).to(dtype)
    ids, tlp = teacher(x, k, 3)
    w = torch.rand(T, generator=g, device="cuda")
    w[torch.rand(T, generator=g, device="cuda") < 0.1] = 0.0
    loss = eqat.distill_topk_fwd(x, ids, tlp, weight=w, tail=tail)
    first = None
    for _ in range(6):
        again, grad = eqat.distill_topk_step(x, ids, tlp, weight=w, tail=tail)
        assert torch.equal(again, loss)
        first = grad if first is None else first
        assert torch.equal(grad, first)
    rows = torch.arange(0, T, 97, device="cuda")
    want_l, want_g = orc.distill_topk(f64(x[rows]), ids[rows].cpu().numpy(), f64(tlp[rows]), f64(w[rows]), 1.0, tail)
    wn = f64(w[rows])
    same(f64(loss[rows]), want_l, wn * 4 * tol(V) + np.abs(want_l) * 2.0 ** -22 + 1e-37, "loss")
    # the bound of check_distill with its largest mass, 1
    rel = 2 * tol(V) + 2.0 ** -20 + 150 * 2.0 ** -23
    same(f64(grad[rows]), want_g, wn[:, None] * 3 * rel + np.abs(want_g) * (HALF[dtype] + 2.0 ** -22) + 1e-37, "gradient")
    want = eqat.token_logprobs(x, ids[:, 0].contiguous(), top_k=k)
    for _ in range(3):
        for a, b in zip(eqat.token_logprobs(x, ids[:, 0].contiguous(), top_k=k), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_distill_in_place_and_padding_left_alone(dtype):
    T, V, ld = 33, 1001, 1024
    wide = torch.randn(T, ld, device="cuda").to(dtype)
    pad = wide[:, V:].clone()
    x = wide[:, :V]
    ids, tlp = teacher(x, 8, 1)
    # same strides, same order of additions: bit for bit
    want = eqat.distill_topk_bwd(x, ids, tlp, torch.ones(T, device="cuda"), tail=True)
    assert want.stride() == x.stride()
    out = torch.full((T, ld), 7.0, dtype=dtype, device="cuda")
    eqat.distill_topk_bwd(x, ids, tlp, torch.ones(T, device="cuda"), tail=True, dlogits=out[:, :V])
    assert torch.equal(out[:, :V], want) and (out[:, V:] == 7.0).all()
    got = eqat.distill_topk_bwd(x, ids, tlp, torch.ones(T, device="cuda"), tail=True, dlogits=x)
    assert got.data_ptr() == x.data_ptr()
    assert torch.equal(x, want) and torch.equal(wide[:, V:], pad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_distill_gradient_of_rows_far_apart(dtype):
    """The last position of each sequence of [B, S, V]: the gradient does not take the
    parent's memory, and is the same bits at any of its strides."""
    for B, S, V in ((5, 64, 1001), (9, 33, 3002), (3, 64, 70001)):
        parent = torch.randn(B, S, V, device="cuda").to(dtype)
        step = 16 // parent.element_size()
        at = max(i for i in range(S) if i * V % step == 0)  # its first row starts on 16 bytes
        x = parent[:, at]
        ids, tlp = teacher(x, 8, 1)
        w = torch.rand(B, device="cuda")
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        loss, grad = eqat.distill_topk_step(x, ids, tlp, weight=w, tail=True)
        assert torch.cuda.max_memory_allocated() - before < 2 * B * (V + step) * x.element_size() + 8192
        check_distill(x, ids, tlp, w, 1.0, True)
        wide = torch.full((B, S * V), 7.0, dtype=dtype, device="cuda")  # logits' own stride
        out = wide[:, :V]
        assert eqat.distill_topk_bwd(x, ids, tlp, w, tail=True, dlogits=out) is out
        assert torch.equal(out, grad) and bool((wide[:, V:] == 7.0).all())
        with pytest.raises(ValueError):
            eqat.distill_topk_bwd(x, ids, tlp, w, dlogits=torch.empty(B, S * V + 1, dtype=dtype, device="cuda")[:, :V])
        eqat.distill_topk_bwd(x, ids, tlp, w, tail=True, dlogits=x)
        assert torch.equal(x, grad)


def test_distill_gradient_beside_the_logits():
    """Logits and gradient as two halves of one buffer's rows; a gradient that overlaps its
    logits is refused."""
    T, V = 40, 1000
    both = torch.randn(T, 2 * V, device="cuda")
    x, g = both[:, :V], both[:, V:]
    ids, tlp = teacher(x, 8, 1)
    w = torch.ones(T, device="cuda")
    want = eqat.distill_topk_bwd(x, ids, tlp, w)
    keep = x.clone()
    eqat.distill_topk_bwd(x, ids, tlp, w, dlogits=g)
    assert torch.equal(g, want) and torch.equal(x, keep)
    with pytest.raises(eqat.EqatError):
        eqat.distill_topk_bwd(both[:-1, :V], ids[1:], tlp[1:], w[1:], dlogits=both[1:, :V])
    assert torch.equal(x, keep)


def test_distill_gradient_matches_differences():
    """The kernel's gradient against central differences of the kernel's own fp32 loss,
    summed along a random direction: h = 2^-4 leaves a third-order error of about
    h^2 |d|^3 / 6 per row and a rounding error of 2 tol / h."""
    T, V, k = 8, 257, 12
    x = make(T, V, torch.float32, 8)
    ids, tlp = teacher(x, k, 2)
    d = torch.nn.functional.normalize(torch.randn(T, V, device="cuda"), dim=1)
    h = 2.0 ** -4
    for tail in (False, True):
        up = eqat.distill_topk_fwd(x + h * d, ids, tlp, tail=tail).double()
        dn = eqat.distill_topk_fwd(x - h * d, ids, tlp, tail=tail).double()
        g = eqat.distill_topk_bwd(x, ids, tlp, torch.ones(T, device="cuda"), tail=tail)
        num, ana = (up - dn) / (2 * h), (g.double() * d.double()).sum(1)
        assert (num - ana).abs().max().item() < h * h / 6 + 2 * tol(V) / h


def test_rows_on_a_side_stream_and_in_a_captured_graph():
    T, V, k = 40, 4099, 9
    x = make(T, V, torch.bfloat16, 3)
    tg = torch.arange(T, device="cuda")
    want = eqat.token_logprobs(x, tg, top_k=k)
    want_l, want_g = eqat.distill_topk_step(x, want[2], want[3], tail=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = eqat.token_logprobs(x, tg, top_k=k)
        l, g = eqat.distill_topk_step(x, got[2], got[3], tail=True)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(l, want_l) and torch.equal(g, want_g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = eqat.token_logprobs(x, tg, top_k=k)
        l, g = eqat.distill_topk_step(x, got[2], got[3], tail=True)
    x.copy_(make(T, V, torch.bfloat16, 4))
    graph.replay()
    torch.cuda.synchronize()
    again = eqat.token_logprobs(x, tg, top_k=k)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    l2, g2 = eqat.distill_topk_step(x, again[2], again[3], tail=True)
    assert torch.equal(l, l2) and torch.equal(g, g2)


def test_rows_past_32_bit_offsets():
    """Rows that start 2^30 elements apart, and one of 2^28 + 3 entries."""
    V, ld = 1001, 1 << 30
    y = make(3, V, torch.bfloat16, 17)
    x = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((3, V), (ld, 1))
    x.copy_(y)
    # rows that start as x's do, on 16 bytes: the order of the sums depends on it
    y = torch.nn.functional.pad(y, (0, 7))[:, :V]
    t = torch.tensor([1, 1000, 500], device="cuda")
    for a, b in zip(eqat.token_logprobs(x, t, top_k=5), eqat.token_logprobs(y, t, top_k=5)):
        assert torch.equal(a, b)
    ids = torch.arange(4, device="cuda").repeat(3, 1)
    tlp = torch.full((3, 4), -2.0, device="cuda")
    want_l, want_g = eqat.distill_topk_step(y, ids, tlp, tail=True)
    loss, grad = eqat.distill_topk_step(x, ids, tlp, tail=True, dlogits=x)
    assert torch.equal(loss, want_l) and torch.equal(grad, want_g)
    del x, grad
    V = (1 << 28) + 3  # equal entries: all sums are whole numbers below 2^24 per thread, but the last
    z = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    z[0, V - 1], z[0, V - 2] = 2.0, 1.0
    S = (V - 2) + np.exp(2.0) + np.exp(1.0)
    for k in (0, 3):
        lp, ent, ids, top = eqat.token_logprobs(z, torch.tensor([V - 1], device="cuda"), top_k=k)
        # ln S near 19.4: three fp32 roundings of it, and 2^-20 of the sums' joins
        assert abs(lp.item() - (2 - np.log(S))) < 1e-5
        assert abs(ent.item() - (np.log(S) - (2 * np.exp(2.0) + np.exp(1.0)) / S)) < 5e-5
    assert ids.tolist() == [[V - 1, V - 2, 0]]
    assert abs(top[0, 2].item() + np.log(S)) < 1e-5


def test_refusals_on_the_device():
    """Refused before anything of their size is allocated or launched."""
    x, t = make(3, 40, torch.float32, 1), torch.zeros(3, dtype=torch.int64, device="cuda")
    tlp = torch.zeros(3, 2, device="cuda")
    for k in (129, -1, 1 << 40):
        with pytest.raises(eqat.EqatError):
            eqat.token_logprobs(x, t, top_k=k)
    for call in [lambda: eqat.token_logprobs(x, None), lambda: eqat.token_logprobs(x, t.int()),
                 lambda: eqat.token_logprobs(x.half(), t), lambda: eqat.distill_topk_fwd(x, None, tlp),
                 lambda: eqat.distill_topk_fwd(x, t[:, None].expand(3, 2).contiguous(), None),
                 lambda: eqat.distill_topk_bwd(x, t[:, None].expand(3, 2).contiguous(), tlp, t),
                 lambda: eqat.distill_topk_step(x, t[:, None].expand(3, 2).contiguous(), tlp, dlogits=x.bfloat16())]:
        with pytest.raises(TypeError):
            call()
    lp, ent, ids, top = eqat.token_logprobs(x[:0], t[:0], top_k=3)
    assert lp.shape == ent.shape == (0,) and ids.shape == top.shape == (0, 3)
    loss, grad = eqat.distill_topk_step(x[:0], ids, top)
    assert loss.shape == (0,) and grad.shape == (0, 40)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_distill_at_the_limits_of_v(dtype):
    """The largest vocabulary, and both sides of the largest one whose slots' bits fit beside
    the wide ring (few long rows); slots at both ends of a row."""
    for V in (524288, 262136, 262137, 262140, 262141):
        x = make(2, V, dtype, V)
        ids, tlp = teacher(x, 6, 1)
        ids[1, 0], ids[1, 1], ids[1, 2] = V - 1, 0, V - 9
        x[1, torch.tensor([0, V - 9, V - 1])] += 9.0
        w = torch.tensor([1.0, 0.5], device="cuda")
        for tail in (False, True):
            check_distill(x, ids, tlp, w, 1.0, tail)
        # rows of another phase: none starts on 16 bytes but the first
        wide = torch.full((2, V + 3), float("nan"), dtype=dtype, device="cuda")
        wide[:, :V] = x
        check_distill(wide[:, :V], ids, tlp, w, 1.0, True)
    with pytest.raises(eqat.EqatError):
        eqat.distill_topk_fwd(make(1, 524289, dtype, 1), ids[:1], tlp[:1])


@pytest.mark.parametrize("tau", [1e-6, 0.05, 30.0, 1e6])
def test_distill_temperatures(tau):
    """2^y below 2^-126 is 0 (ex2 flushes it), before it is multiplied by 1 / (tau S) or, outside
    the slots, by at most that and as much again for the teacher's rest (S >= 1, the largest
    entry's term): a gradient is off by up to 2^-125 / tau for that alone, more than 1e-37
    where tau is small."""
    x = make(6, 4097, torch.float32, 1)
    ids, tlp = teacher(x, 20, 3, tau)
    for tail in (False, True):
        check_distill(x, ids, tlp, None, tau, tail, least=1e-37 + 2.0 ** -125 / tau)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 9])
def test_many_rows_within_a_vector(V, dtype):
    """Rows that share their 16 bytes with their neighbours, which other blocks take: the
    gradient in place, the columns past V as they were."""
    T, k = 3000, min(V, 3)
    for ld in (V, V + 1):
        x = make(T, V, dtype, V, ld)
        t = torch.arange(T, device="cuda") % V
        check_logprobs(x, t, k)
        check_logprobs(x, t, 0)
        ids, tlp = teacher(x, k, 5)
        w = torch.rand(T, device="cuda")
        w[::7] = 0.0
        for tail in (False, True):
            _, want = check_distill(x, ids, tlp, w, 1.0, tail)
            buf = torch.full((T, ld), 3.0, dtype=dtype, device="cuda")
            buf[:, :V] = x
            eqat.distill_topk_bwd(buf[:, :V], ids, tlp, w, tail=tail, dlogits=buf[:, :V])
            assert torch.equal(buf[:, :V], want) and bool((buf[:, V:] == 3.0).all())
