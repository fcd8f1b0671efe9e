"""A layer of experts through the products, the clip, the optimizer step and
the block-scaled product, as a training loop and a server use them together;
and the products under concurrent callers.

Every stage is checked against the float64 oracle on the GPU's own inputs of
that stage, so that no error passes from one tolerance into the next:
    products    (len + 2) 2^-24 S + half a bf16 step, S the sum of magnitudes
    clip        dw scaled by max_norm / norm: two fp32 roundings, and half a
                step of the gradient's type
    step        the momentum against the oracle's recurrence (relative error
                <= 1e-6, the step's own measure); the parameters bit by bit
                against the step on matrices of their own.  (An expert of 60
                rows has a gradient of rank 60 at most: the other directions
                hold only the gradient's rounding, about 2^-9, which five
                iterations of slope 3.4445 raise to 485 * 2^-9, so the result
                in them is the products' rounding and no oracle's.)
    block-scaled product against the dequantised operands: half a bf16 step
                and 128 * 2^-13 of each block's largest product
"""
import threading

import numpy as np
import pytest
import torch

from oracle import blocks as ob
from oracle import experts as oe
from oracle import muon as orc
from tests.gpu_helpers import rel

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(rng, shape, dtype=BF, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).to(DEV)


def within(got, ref, mag, length, bf16, what):
    tol = (length + 2) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 1e-37
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol * (1 + 1e-6)), (what, float((err / tol).max()))


@pytest.mark.parametrize("grad_dtype", [BF, F32], ids=["bf16", "f32"])
def test_training_steps(lib, grad_dtype):
    """Two optimizer steps of y = w[e] x with loss 0.5 |y - target|^2, two
    microbatches each: the second adds to the first's weight gradients; then
    the experts' products in 8 bits with the updated weights."""
    rng = np.random.default_rng(31)
    experts, tokens, n, k = 4, 210, 136, 264
    w = normal(rng, (experts, n, k), BF, 0.05)
    mom = [torch.zeros(n, k, dtype=F32, device=DEV) for _ in range(experts)]
    m_ref = [np.zeros((n, k)) for _ in range(experts)]
    hp = dict(lr=0.02, momentum=0.95, nesterov=True, ns_steps=5, weight_decay=0.1)
    for step in range(2):
        dw = torch.empty(experts, n, k, dtype=grad_dtype, device=DEV)
        for micro, off in enumerate(([0, 60, 60, 131, 205], [0, 3, 100, 150, 210])):
            offs = torch.tensor(off, dtype=torch.int32, device=DEV)
            x, target = normal(rng, (tokens, k)), normal(rng, (tokens, n))
            y = lib.dmuon_expert_matmul(x, w, offs, out=target.clone())   # rows of no expert: no loss
            dy = y - target
            dx = torch.zeros(tokens, k, dtype=BF, device=DEV)
            lib.dmuon_expert_input_grad(dy, w, offs, out=dx)
            old = f64(dw) if micro else None
            lib.dmuon_expert_weight_grad(dy, x, offs, out=dw, accumulate=micro > 0)
            X, W, DY = f64(x), f64(w), f64(dy)
            a = np.abs
            within(y, oe.expert_matmul(X, W, off, f64(target)), oe.expert_matmul(a(X), a(W), off, a(f64(target))), k,
                   True, "y")
            zero = np.zeros((tokens, k))
            within(dx, oe.expert_input_grad(DY, W, off, zero), oe.expert_input_grad(a(DY), a(W), off, zero), n, True,
                   "dx")
            within(dw, oe.expert_weight_grad(DY, X, off, old),
                   oe.expert_weight_grad(a(DY), a(X), off, None if old is None else a(old)), 98, grad_dtype == BF, "dw")
        grads = [dw[e] for e in range(experts)]
        before = f64(dw)
        total = lib.dmuon_clip_grad_norm(grads, 1.0)
        norm = np.linalg.norm(before)
        assert abs(float(total[0]) - norm) <= 1e-6 * norm and norm > 1.0
        after, want = f64(dw), before / (norm + 1e-6)
        eps = 2.0 ** -8 if grad_dtype == BF else 2.0 ** -22
        assert np.all(np.abs(after - want) <= (eps + 1e-6) * np.abs(want) + 1e-37)
        own = [[w[e].clone() for e in range(experts)], [g.clone() for g in grads], [m.clone() for m in mom]]
        lib.dmuon_step([w[e] for e in range(experts)], grads, mom, **hp)
        lib.dmuon_step(*own, **hp)
        torch.cuda.synchronize()
        for e in range(experts):
            m_ref[e] = orc.muon_step(f64(w[e]), after[e], m_ref[e], ns_backend="gram", param_dtype="f32", **hp)[1]
            assert rel(f64(mom[e]), m_ref[e]) <= 1e-6, (step, e)
            assert bool(torch.isfinite(w[e]).all()) and torch.equal(w[e], own[0][e])
    wq, ws, _, _ = lib.dmuon_quantize_blocks(w, block_rows=128)
    xq, xs, _, _ = lib.dmuon_quantize_blocks(x)
    y8 = lib.dmuon_block_matmul(xq, xs, wq, ws, block_rows=128, offsets=offs, out=target.clone())
    X = ob.dequantize(f64(xq.float()), f64(xs), 1)
    for e, lo, hi in oe.spans(off, tokens):
        B = ob.dequantize(f64(wq[e].float()), f64(ws[e]), 128)
        ref = X[lo:hi] @ B.T
        tol = 2.0 ** -8 * np.abs(ref) + 1e-37
        for c in range(0, k, 128):
            tol = tol + 128 * 2.0 ** -13 * np.outer(np.abs(X[lo:hi, c:c + 128]).max(1), np.abs(B[:, c:c + 128]).max(1))
        assert np.all(np.abs(f64(y8[lo:hi]) - ref) <= tol * (1 + 1e-6)), e


def test_clip_folded_into_the_step(lib):
    """The clip's coefficients read by the step instead of a pass over the
    experts' fp32 gradients."""
    rng = np.random.default_rng(32)
    experts, tokens, n, k = 3, 90, 64, 96
    off = [0, 30, 60, 90]
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, dy, w = normal(rng, (tokens, k)), normal(rng, (tokens, n)), normal(rng, (experts, n, k), BF, 0.05)
    dw = lib.dmuon_expert_weight_grad(dy, x, offs, out_dtype=F32)
    coef = lib.dmuon_clip_coefficients([dw[e] for e in range(experts)], 1.0)
    g = f64(dw) / np.linalg.norm(f64(dw))
    mom = [torch.zeros(n, k, dtype=F32, device=DEV) for _ in range(experts)]
    hp = dict(lr=0.02, momentum=0.95, nesterov=True, ns_steps=5, weight_decay=0.0)
    own = [[w[e].clone() for e in range(experts)], [dw[e].clone() for e in range(experts)], [m.clone() for m in mom]]
    scale = dict(grad_scale=coef, grad_scale_index=[0] * experts)
    lib.dmuon_step([w[e] for e in range(experts)], [dw[e] for e in range(experts)], mom, **scale, **hp)
    lib.dmuon_step(*own, **scale, **hp)
    for e in range(experts):
        m = orc.muon_step(f64(w[e]), g[e], np.zeros((n, k)), ns_backend="gram", param_dtype="f32", **hp)[1]
        assert rel(f64(mom[e]), m) <= 1e-5
        assert bool(torch.isfinite(w[e]).all()) and torch.equal(w[e], own[0][e])


# tile counts of the 256 x 256 kernels that leave 16, 112 and 208 tiles behind
# a whole round of 256: parts of 64 and 128 rows, and whole ones; and 48 tiles
# where the offsets could need 224
LEFT = [(4300, 4096, 72, [0, 4200]), (5600, 4096, 72, [0, 2700, 2700, 5600]), (7250, 4096, 72, [3, 7245]),
        (2100, 4096, 72, [0, 0, 0, 0, 0, 0, 600])]


@pytest.mark.parametrize("case", LEFT, ids=lambda c: f"{c[0]}-{len(c[3]) - 1}")
def test_left_over_tiles(lib, case):
    """Against float64 products on the GPU."""
    rng = np.random.default_rng(33)
    tokens, n, k, off = case
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    experts = len(off) - 1
    x, w, wt = normal(rng, (tokens, k)), normal(rng, (experts, n, k)), normal(rng, (experts, k, n))
    qx, sx, _, _ = lib.dmuon_quantize_blocks(x)
    qw, sw, _, _ = lib.dmuon_quantize_blocks(w, block_rows=128)
    keep = normal(rng, (tokens, n))
    y, dx, y8 = keep.clone(), keep.clone(), keep.clone()
    lib.dmuon_expert_matmul(x, w, offs, out=y)
    lib.dmuon_expert_input_grad(x, wt, offs, out=dx)       # the same sums from the other layout
    lib.dmuon_block_matmul(qx, sx, qw, sw, block_rows=128, offsets=offs, out=y8)
    X8 = lib.dmuon_dequantize_blocks(qx, sx, dtype=F32).double()
    W8 = lib.dmuon_dequantize_blocks(qw, sw, block_rows=128, dtype=F32).double()
    for got, A, B in ((y, x.double(), w.double()), (dx, x.double(), wt.double().transpose(1, 2).contiguous()),
                      (y8, X8, W8)):
        out = torch.ones(tokens, dtype=torch.bool, device=DEV)
        for e, lo, hi in oe.spans(off, tokens):
            a, b = A[lo:hi], B[e].t().contiguous()
            ref, mag = a @ b, a.abs() @ b.abs()
            tol = 2.0 ** -8 * ref.abs() + (k + 2) * 2.0 ** -24 * mag
            if got is y8:
                tol = tol + 128 * 2.0 ** -13 * torch.outer(a.abs().amax(1), b.abs().amax(0))
            assert bool(((got[lo:hi].double() - ref).abs() <= tol * (1 + 1e-6)).all())
            out[lo:hi] = False
        assert torch.equal(got[out], keep[out])


def test_more_experts_than_the_large_tiles_hold(lib):
    """1030 experts, one row each and some none."""
    rng = np.random.default_rng(34)
    off = np.concatenate([[0], np.cumsum(np.arange(1030) % 3 != 0)]).astype(int).tolist()
    tokens, n, k = off[-1] + 5, 40, 48
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, w, dy = normal(rng, (tokens, k)), normal(rng, (1030, n, k)), normal(rng, (tokens, n))
    X, W, DY = f64(x), f64(w), f64(dy)
    a = np.abs
    y = torch.zeros(tokens, n, dtype=BF, device=DEV)
    dx = torch.zeros(tokens, k, dtype=BF, device=DEV)
    within(lib.dmuon_expert_matmul(x, w, offs, out=y), oe.expert_matmul(X, W, off, f64(y) * 0),
           oe.expert_matmul(a(X), a(W), off, np.zeros((tokens, n))), k, True, "y")
    within(lib.dmuon_expert_input_grad(dy, w, offs, out=dx), oe.expert_input_grad(DY, W, off, np.zeros((tokens, k))),
           oe.expert_input_grad(a(DY), a(W), off, np.zeros((tokens, k))), n, True, "dx")
    within(lib.dmuon_expert_weight_grad(dy, x, offs, out_dtype=F32), oe.expert_weight_grad(DY, X, off),
           oe.expert_weight_grad(a(DY), a(X), off), 1, False, "dw")


@pytest.mark.parametrize("dtype,n,k", [(BF, 2048, 2048), (BF, 72, 40), (F32, 65, 33)])
def test_accumulate_leaves_experts_without_rows(lib, dtype, n, k):
    """Bit for bit, a negative zero among them."""
    rng = np.random.default_rng(36)
    x, dy = normal(rng, (20, k), dtype), normal(rng, (20, n), dtype)
    dw = torch.full((4, n, k), -0.0, dtype=dtype, device=DEV)
    dw[2, 0, 0] = float("inf")
    offs = torch.tensor([0, 0, 7, 7, 20], dtype=torch.int32, device=DEV)
    lib.dmuon_expert_weight_grad(dy, x, offs, out=dw, accumulate=True)
    assert bool(torch.signbit(dw[0]).all()) and bool(torch.isinf(dw[2, 0, 0]))
    dw[2, 0, 0] = -0.0
    assert bool(torch.signbit(dw[2]).all())
    lib.dmuon_expert_weight_grad(dy, x, offs, out=dw)
    assert not bool(dw[0].any()) and not bool(dw[2].any()) and bool(dw[1].any())


def test_concurrent_callers(lib):
    """Four threads with a stream each: every result equals the one of the
    same call made alone."""
    rng = np.random.default_rng(35)
    off = [0, 40, 40, 300]
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    data = []
    for _ in range(4):
        x, w, dy = normal(rng, (300, 520)), normal(rng, (3, 200, 520)), normal(rng, (300, 200))
        data.append((x, w, dy))

    def calls(x, w, dy, stream=None):
        outs = [torch.zeros(300, 200, dtype=BF, device=DEV), torch.zeros(300, 520, dtype=BF, device=DEV)]
        torch.cuda.synchronize()
        for _ in range(10):
            lib.dmuon_expert_matmul(x, w, offs, out=outs[0], stream=stream)
            lib.dmuon_expert_input_grad(dy, w, offs, out=outs[1], stream=stream)
            dw = lib.dmuon_expert_weight_grad(dy, x, offs, out_dtype=F32, stream=stream)
            q, s, _, _ = lib.dmuon_quantize_blocks(x, stream=stream)
            b, t, _, _ = lib.dmuon_quantize_blocks(w[0], block_rows=128, stream=stream)
            z = lib.dmuon_block_matmul(q, s, b, t, block_rows=128, stream=stream)
        return outs + [dw, z]

    want = [calls(*d) for d in data]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got[i] = calls(*data[i], stream=stream)
            stream.synchronize()
        except Exception as e:      # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
