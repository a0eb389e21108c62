"""The E2E-QP step of a quantized output projection (teacher's alternatives, packed
forward, distillation, scales' gradient, AdamW), checked against the same chain of
oracles: the kernels' own bf16 logits are compared with the oracle's product, and the
loss, dX, ds and the updated s with what the oracles make of them."""
import numpy as np
import pytest
import torch

import weight_quantization_aware_b200 as eqat
from oracle import rows
from parity import TOL_GEMM, TOL_RED, assert_close, to_np
from weight_quantization_aware_b200 import e2eqp, synthetic

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_quantization_aware_b200 import build
    build.build()
    eqat.load_library()
    yield
    assert eqat.device_error() == 0


@pytest.mark.parametrize("T", [5, 96])
@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
def test_head_step(orc, T, tail):
    V, K, k, bits, g = 1032, 256, 12, 4, 64
    d = synthetic.draw_linear(np.random.default_rng(7), T, V, K, 0.1, "bf16")
    X, W = d["X"].cuda(), d["W"].cuda()
    s, z = eqat.minmax_init(W, bits, g)
    codes, zq = eqat.pack_codes(W, s, z, bits, g)
    teacher = (X.float() @ W.float().t()).to(torch.bfloat16)
    ids, tlp = e2eqp.teacher_alternatives(teacher, k, 1.5)
    _, _, w_ids, w_tlp = rows.token_logprobs(to_np(teacher), np.full(T, -1), k, 1.5)
    assert np.array_equal(to_np(ids), w_ids) and np.abs(to_np(tlp) - w_tlp).max() < 1e-5

    head = e2eqp.QuantHead(codes, zq, s.clone())
    cfg = e2eqp.E2EQPConfig(bits=bits, group=g, temperature=1.5, tail=tail)
    Y = eqat.dq_linear_fwd(X, codes, zq, s, bits, g)  # the step's logits, before they are overwritten
    loss, dX = e2eqp.e2eqp_head_step(head, X, ids, tlp, cfg, 1)

    Xn, cn, zn, sn = synthetic.as_f32_numpy(d["X"]), to_np(codes), to_np(zq), to_np(s)
    assert_close(to_np(Y), orc.dq_linear_fwd(Xn, cn, zn, sn, bits, g), TOL_GEMM, "logits")
    want_l, want_g = rows.distill_topk(to_np(Y), to_np(ids), to_np(tlp), np.full(T, 1.0 / T), 1.5, tail)
    assert np.abs(to_np(loss) - want_l).max() <= 1e-5 * max(1.0, np.abs(want_l).max())
    dYn = torch.from_numpy(want_g.astype(np.float32)).to(torch.bfloat16).float().numpy()
    dX_ref, ds_ref = orc.dq_linear_bwd_s(Xn, cn, zn, sn, dYn, bits, g)
    # dY is rounded to bf16 on both sides, by at most 2^-8 apart where the fp32 values differ
    assert_close(to_np(dX), dX_ref, TOL_GEMM, "dX")
    dX2, ds = eqat.dq_linear_bwd_s(X, codes, zq, s, torch.from_numpy(dYn).to(torch.bfloat16).cuda(), bits, g)
    assert_close(to_np(ds), ds_ref, TOL_RED, "ds")
    p_ref, _, _ = orc.adamw(sn, ds_ref.astype(np.float32), np.zeros_like(sn), np.zeros_like(sn), 2e-5, 0.9, 0.999, 1e-8, 0.0, 1)
    # the first AdamW step moves every s by lr times the sign of its gradient
    moved = to_np(head.s) - sn
    sure = np.abs(ds_ref) > 0.05 * np.abs(ds_ref).max()
    assert np.array_equal(np.sign(moved)[sure], np.sign(p_ref - sn)[sure])
    assert np.abs(moved).max() <= 2.1e-5


def test_head_steps_of_many_then_few_tokens():
    """The head's workspace follows the token count: a narrow layer needs more for few
    tokens (partial sums) than for many (W-hat)."""
    V, K, bits, g = 8, 128, 2, 64
    d = synthetic.draw_linear(np.random.default_rng(8), 40, V, K, 0.1, "bf16")
    X, W = d["X"].cuda(), d["W"].cuda()
    s, z = eqat.minmax_init(W, bits, g)
    codes, zq = eqat.pack_codes(W, s, z, bits, g)
    ids, tlp = e2eqp.teacher_alternatives((X.float() @ W.float().t()).to(torch.bfloat16), 4)
    cfg = e2eqp.E2EQPConfig(bits=bits, group=g)
    head = e2eqp.QuantHead(codes, zq, s.clone())
    for step, T in enumerate((40, 8, 3, 40), 1):
        alone = e2eqp.QuantHead(codes, zq, head.s.clone())
        want, want_dx = e2eqp.e2eqp_head_step(alone, X[:T], ids[:T], tlp[:T], cfg, 1)
        loss, dX = e2eqp.e2eqp_head_step(head, X[:T], ids[:T], tlp[:T], cfg, step)
        assert torch.equal(loss, want) and torch.equal(dX, want_dx)


def test_head_step_without_tokens():
    """A batch whose tokens are all masked away: no loss, dX of no rows, a gradient of 0 for
    the scales (AdamW goes on by its moments)."""
    V, K, k, bits, g = 136, 128, 4, 2, 64
    d = synthetic.draw_linear(np.random.default_rng(9), 40, V, K, 0.1, "bf16")
    X, W = d["X"].cuda(), d["W"].cuda()
    s, z = eqat.minmax_init(W, bits, g)
    codes, zq = eqat.pack_codes(W, s, z, bits, g)
    teacher = (X.float() @ W.float().t()).to(torch.bfloat16)
    ids, tlp = e2eqp.teacher_alternatives(teacher[:0], k)
    assert ids.shape == (0, k) and tlp.shape == (0, k)
    cfg = e2eqp.E2EQPConfig(bits=bits, group=g)
    head = e2eqp.QuantHead(codes, zq, s.clone())
    loss, dX = e2eqp.e2eqp_head_step(head, X[:0], ids, tlp, cfg, 1)
    assert loss.shape == (0,) and dX.shape == (0, K)
    assert torch.equal(head.s, s) and not head.moments[0].any() and not head.moments[1].any()
    ids, tlp = e2eqp.teacher_alternatives(teacher, k)
    e2eqp.e2eqp_head_step(head, X, ids, tlp, cfg, 2)
    m, v, now = head.moments[0].clone(), head.moments[1].clone(), head.s.clone()
    assert m.any()
    e2eqp.e2eqp_head_step(head, X[:0], ids[:0], tlp[:0], cfg, 3)
    # one fp32 rounding each of 0.9 m and 0.999 v, and of beta itself
    assert torch.allclose(head.moments[0], 0.9 * m, rtol=2.0 ** -22, atol=0)
    assert torch.allclose(head.moments[1], 0.999 * v, rtol=2.0 ** -22, atol=0)
    assert not torch.equal(head.s, now)
