"""The top logits and the distillation loss on many rows (a CTA works on several), and on rows whose
logits are far from zero."""

import numpy as np
import pytest
import torch

from tests.test_gpu_distill import BF16, F32, INF, NAN, check_top, make

pytestmark = pytest.mark.gpu


def reference(x, tv, ti, temp, w, g):
    """float64 (loss, gradient, p, Q), logits relative to their row's maximum."""
    x, tv = x.double().cpu().numpy(), tv.double().cpu().numpy()
    ti = ti.cpu().numpy()
    n, v = x.shape
    loss, grad, p, Q = np.zeros(n), np.zeros((n, v)), np.zeros((n, v)), np.zeros((n, v))
    for i in range(n):
        on = (ti[i] >= 0) & (tv[i] > -np.inf)
        if w[i] == 0 or not on.any():
            continue
        d = (x[i] - x[i].max()) / temp
        logz = np.log(np.exp(d).sum())
        p[i] = np.exp(d - logz)
        t = (tv[i][on] - tv[i][on].max()) / temp
        logq = t - np.log(np.exp(t).sum())
        np.add.at(Q[i], ti[i][on], np.exp(logq))
        loss[i] = w[i] * (np.exp(logq) * (logq - (d[ti[i][on]] - logz))).sum()
        grad[i] = g[i] * w[i] * (p[i] - Q[i]) / temp
    return loss, grad, p, Q


def check(loss, grad, ref, size, w, g, temp, dtype, extra=0.0):
    """Exponents are off by 2^-22 of their terms' size, exp2 and the float32 sums by 2^-20 of the
    result; `extra` is a further relative error of p."""
    rl, rg, p, Q = ref
    rel = 2.0 ** -20 + 2.0 ** -22 * size
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= 4 * rel * np.maximum(np.abs(w), 1) * (1 + np.abs(rl)))
    err = np.abs(grad.double().cpu().numpy() - rg)
    tol = (np.abs(g * w) / temp)[:, None] * ((rel + extra) * (p + Q))
    assert np.all(err <= tol + (2.0 ** -8 * np.abs(rg) if dtype == BF16 else 0) + 1e-37)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,v", [(1000, 3001), (700, 60001)])   # short rows and long ones
def test_distill_many_rows(lib, cuda_device, dtype, n, v):
    """Several rows a CTA, some of weight 0 (whose logits are not read) and some without entries
    among them: loss alone, loss and gradient, the two calls, and in place."""
    gen = torch.Generator().manual_seed(n)
    x, tv, ti, w, gl = make(gen, n, v, 24, dtype, cuda_device)
    w[torch.rand(n, generator=gen).to(cuda_device) < 0.3] = 0.0
    ti[torch.rand(n, generator=gen).to(cuda_device) < 0.2] = -1
    ti[5::7, 3] = ti[5::7, 0]
    hw, hg = w.double().cpu().numpy(), gl.double().cpu().numpy()
    ref = reference(x, tv, ti, 2.0, hw, np.ones(n))
    x[w == 0] = NAN
    size = 40.0
    loss, lse = lib.gptq_distill_loss(x, tv, ti, temperature=2.0, weights=w)
    dx = lib.gptq_distill_backward(x, lse, tv, ti, gl, temperature=2.0, weights=w)
    check(loss, dx, (ref[0], ref[1] * hg[:, None], *ref[2:]), size, hw, hg, 2.0, dtype)
    loss2, dx2 = lib.gptq_distill_loss_grad(x, tv, ti, temperature=2.0, weights=w)
    check(loss2, dx2, ref, size, hw, np.ones(n), 2.0, dtype)
    same = x.clone()
    loss3, dx3 = lib.gptq_distill_loss_grad(same, tv, ti, temperature=2.0, weights=w, dlogits=same)
    assert torch.equal(loss3, loss2) and torch.equal(dx3, dx2)
    same = x.clone()
    dx4 = lib.gptq_distill_backward(same, lse, tv, ti, gl, temperature=2.0, weights=w, dlogits=same)
    assert torch.equal(dx4, dx)
    lib.gptq_async_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("temp", [1.0, 0.5, 3.0])
def test_distill_backward_far_from_zero(lib, cuda_device, dtype, temp):
    """Rows whose logits are all the type's lowest value (a mask that leaves nothing), or lie far
    from zero: the log-sum-exp that the backward call is given is rounded to float32, or is
    infinite, but the gradient is that of the row."""
    gen = torch.Generator().manual_seed(3)
    v = 5003
    x, tv, ti, w, gl = make(gen, 12, v, 16, dtype, cuda_device, short=False)
    low = torch.finfo(dtype).min
    x[0] = low
    x[1] = low
    x[1, 100:200] = low / 2
    x[2] = torch.finfo(dtype).max
    x[3] = (x[3].float() * 2.0 ** 20).to(dtype)
    x[4] = (x[4].float() + 1e5).to(dtype)
    x[5] = -1e30
    x[6] = 3000.0
    x[7] = (x[7].float() - 1500.0).to(dtype)
    x[8] = -70000.0
    x[8, 1:400:2] = -70000.0 + 512
    ti[:9] = torch.arange(90, 106, dtype=torch.int32)
    hw, hg = w.double().cpu().numpy(), gl.double().cpu().numpy()
    ref = reference(x, tv, ti, temp, hw, hg)
    loss, lse = lib.gptq_distill_loss(x, tv, ti, temperature=temp, weights=w)
    dx = lib.gptq_distill_backward(x, lse, tv, ti, gl, temperature=temp, weights=w)
    # up to 1024 the rounding of Z, 2^-24 of it, is left in p; entries so far below the maximum that
    # the loss itself is out of range are not compared
    rl = ref[0]
    rows = [i for i in range(12) if abs(rl[i]) < 1e6]
    assert {0, 2, 4, 5, 6, 7, 8} <= set(rows)
    d = x.double().cpu().numpy()
    size = ((d.max(1) - np.sort(d, 1)[:, 0]) / temp).clip(0, 2000)
    size = np.maximum(size, 30)
    # teacher values are below 16; logits at the entries count relative to the row's maximum
    for i in rows:
        check(loss[i:i + 1], dx[i:i + 1], [a[i:i + 1] for a in ref], size[i], hw[i:i + 1], hg[i:i + 1],
              temp, dtype, extra=2.0 ** -13)
    same = x.clone()
    out = lib.gptq_distill_backward(same, lse, tv, ti, gl, temperature=temp, weights=w, dlogits=same)
    assert torch.equal(out, dx)
    lib.gptq_async_status()


@pytest.mark.parametrize("rows,vocab,dtype", [(400, 2000, BF16), (50, 1003, F32), (3, 1500, BF16)])
def test_top_logits_of_few_pieces(lib, cuda_device, rows, vocab, dtype):
    """Fewer 16-byte pieces in a row than k, so that most threads see no element, and more elements
    than are held as candidates."""
    gen = torch.Generator().manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=gen) * 3).to(dtype).to(cuda_device)
    x[1, 5:900] = -INF
    check_top(lib, x, 256)
