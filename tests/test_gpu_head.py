"""Cross entropy and distillation through a stored vocabulary projection on
the GPU against the fp64 oracle, every output compared; then a training step
of adapters through a block and the projection.

Bounds (u = 2^-24):
  z      (cols + 2 ngroups + 3) u sum |h| |q - z| s / T, as the product with
         adapters
  exp    off by at most 4 u (|z - lse| + 2) of itself (the argument's rounding
         and the instruction's), so the sum of exponentials by the average of
         that over the softmax, and (40 + tiles / 64) u for its additions
  lse    the largest z error, the sum's, and 4 u (|lse| + 1)
  loss   sum p times (z's error + lse's + 4 u of the sizes), p itself off by
         8 u (|log p| + 2) of itself
  dh     each probability off by z's and lse's errors and exp's, and each
         p - target rounded to fp16 (2^-11 of it, 2^-25 below 2^-14), against
         |W_hat|; W_hat's own rounding against |p - target|; (rows + pieces + 2)
         u for the sum; half an fp16 step of the result
"""
import numpy as np
import pytest

import oracle
from test_gpu_adapters import U, Layer, _adapters, _cuda, half_step16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import post_weight_quantization_02_amd as gq
    return torch, gq


def _hidden(rng, L, m, sure=1.0):
    """Hidden states whose tokens lean towards a few entries."""
    h = rng.standard_normal((m, L.cols)) * 2
    near = rng.integers(0, L.rows, m)
    size = (L.W ** 2).sum(1)[near, None]
    return (h + sure * rng.random((m, 1)) * 12 * L.W[near] / size).astype(np.float16), near


def _labels(rng, m, rows, near):
    y = np.where(rng.random(m) < 0.5, near, rng.integers(0, rows, m))
    y[rng.random(m) < 0.15] = -100
    if m > 3:
        y[1], y[2], y[3] = rows, rows - 1, -1
    return y.astype(np.int32)


def _teacher(rng, m, top, rows, near):
    idx = rng.integers(0, rows, (m, top))
    idx[:, 0] = near
    if top > 2:
        idx[0, 1] = idx[0, 0]             # an index twice
    logits = (rng.standard_normal((m, top)) * 4).astype(np.float32)
    logits[rng.random((m, top)) < 0.1] = -np.inf
    idx[rng.random((m, top)) < 0.1] = -1
    idx[rng.random((m, top)) < 0.03] = rows
    if m > 4:
        idx[3] = -1                       # no entry by index,
        logits[4] = -np.inf               # by logit
        logits[1] *= 30                   # probabilities that underflow
    return idx.astype(np.int32), logits


def _compare(env, L, h, index, logits, T, dloss, got):
    """The three outputs and dh against the oracle within the bounds above."""
    loss, lse, zk, dh = (t.cpu().numpy().astype(np.float64) for t in got)
    m = len(h)
    rl, rlse, rzk, z = oracle.head_loss(h, L.W, index, logits, T)
    p, part = oracle.head_targets(index, logits, L.rows, T)
    ez = (L.cols + 2 * L.ng + 3) * U * (np.abs(h.astype(np.float64)) @ np.abs(L.W).T) / T
    soft = np.exp(z - rlse[:, None])
    tiles = -(-L.rows // 128)
    elog = 4 * U * (np.abs(z - rlse[:, None]) + 2)
    tlse = ez.max(1) + (soft * elog).sum(1) + (40 + tiles / 64) * U + 4 * U * (np.abs(rlse) + 1)
    assert np.all(np.abs(lse - rlse) <= tlse), float(np.abs(lse - rlse).max())
    idx = np.clip(np.asarray(index, np.int64).reshape(m, -1), 0, L.rows - 1)
    ezk = np.where(part, np.take_along_axis(ez, idx, 1), 0)
    assert np.all(np.abs(zk.reshape(m, -1) - rzk) <= ezk + 2 * U * np.abs(rzk))
    lp = np.log(np.where(p > 0, p, 1))
    ep = 8 * U * (np.abs(lp) + 2) if logits is not None else 0 * lp
    size = np.abs(lp) + np.abs(rzk) + np.abs(rlse)[:, None]
    tloss = np.where(part, p * (ezk + tlse[:, None] + 16 * U * size)
                     + p * ep * np.abs(lp - rzk + rlse[:, None]), 0).sum(1) + p.shape[1] * U * size.max(1)
    # probabilities below the smallest normal are flushed: exp(-87) of the rest
    assert np.all(np.abs(loss - rl) <= tloss + 1e-36), float(np.abs(loss - rl).max())
    out = ~part.any(1)
    assert not loss[out].any() and not dh[out].any() and not zk.reshape(m, -1)[~part].any()

    dz = oracle.head_dz(z, index, logits, T)
    w = np.abs(dloss.astype(np.float64))[:, None] / T
    ref = (dloss.astype(np.float64)[:, None] / T) * (dz @ L.W)
    es = soft * (ez + tlse[:, None] + elog)
    for t in range(m):
        for k in np.nonzero(part[t])[0]:
            es[t, idx[t, k]] += p[t, k] * (ep[t, k] + 4 * U)
    es[out] = 0
    edz = es + (np.abs(dz) + es) * 2.0 ** -11 + np.where(out[:, None], 0, 2.0 ** -25)
    tol = edz @ np.abs(L.W) + (np.abs(dz) + edz) @ (np.abs(L.W) * (2.0 ** -11 + 2 * U) + 2.0 ** -25)
    tol += (L.rows + 130) * U * (np.abs(dz) @ np.abs(L.W))
    tol = w * tol * (1 + 2.0 ** -20)
    tol += half_step16(np.abs(ref) + tol)
    err = np.abs(dh - ref)
    assert np.all(err <= tol), (float(err.max()), int((err > tol).sum()))


def _run(env, L, h, index, logits, T, dloss):
    torch, gq = env
    hd, i, g = _cuda(env, h), _cuda(env, index), _cuda(env, dloss)
    if logits is None:
        loss, lse, zk = gq.head_loss(hd, *L.args, i)
        dh = gq.head_loss_backward(hd, *L.args, i, lse, zk, g)
    else:
        t = _cuda(env, logits)
        loss, lse, zk = gq.head_distill(hd, *L.args, i, t, T)
        dh = gq.head_distill_backward(hd, *L.args, i, t, T, lse, zk, g)
    torch.cuda.synchronize()
    return loss, lse, zk, dh


def _case(env, m, rows, cols, bits, g, top, T, seed):
    L = Layer(env, rows, cols, bits, g, seed)
    rng = np.random.default_rng(seed + 1)
    h, near = _hidden(rng, L, m)
    index, logits = (_labels(rng, m, rows, near), None) if top == 0 else _teacher(rng, m, top, rows, near)
    dloss = (rng.standard_normal(m) * 4).astype(np.float32)
    _compare(env, L, h, index, logits, T, dloss, _run(env, L, h, index, logits, T, dloss))


SHAPES = [(1, 1, 128, 4, 128), (1, 300, 256, 4, 128), (5, 257, 128, 8, 128), (17, 1000, 256, 4, 0),
          (129, 511, 384, 4, 256), (130, 640, 256, 8, 128), (300, 1025, 256, 4, 128)]


@pytest.mark.parametrize("m,rows,cols,bits,g", SHAPES)
def test_cross_entropy(env, m, rows, cols, bits, g):
    _case(env, m, rows, cols, bits, g, 0, 1.0, seed=m + rows)


@pytest.mark.parametrize("m,rows,cols,bits,g", SHAPES)
@pytest.mark.parametrize("top,T", [(1, 1.0), (5, 2.0), (64, 0.7), (256, 4.0)])
def test_distillation(env, m, rows, cols, bits, g, top, T):
    _case(env, m, rows, cols, bits, g, top, T, seed=m + rows + top)


def test_several_pieces_of_the_vocabulary(env):
    """2100 x 40011 probabilities: three pieces of the vocabulary, the last
    one ragged; then 9001 x 8192 weights: two pieces. The largest tiles too,
    in the products and the gradient."""
    _case(env, 2100, 40011, 128, 4, 128, 0, 1.0, seed=1)
    _case(env, 3, 9001, 8192, 4, 128, 16, 2.0, seed=2)


def test_more_tokens_than_one_pass(env):
    """8192 tokens a pass: 8200, sampled where the passes meet."""
    torch, gq = env
    L = Layer(env, 600, 128, 4, 128, 1)
    rng = np.random.default_rng(2)
    m = 8200
    h, near = _hidden(rng, L, m)
    y = _labels(rng, m, 600, near)
    g = rng.standard_normal(m).astype(np.float32)
    got = _run(env, L, h, y, None, 1.0, g)
    pick = np.r_[0:40, 8150:8200]
    p = torch.from_numpy(pick).cuda()
    _compare(env, L, h[pick], y[pick], None, 1.0, g[pick], [t[p] for t in got])


def test_full_vocabulary_shape(env):
    """32000 x 4096, 48 tokens."""
    _case(env, 48, 32000, 4096, 4, 128, 0, 1.0, seed=3)


def test_ignored_tokens_may_hold_anything(env):
    torch, gq = env
    L = Layer(env, 300, 256, 4, 128, 1)
    rng = np.random.default_rng(4)
    h, near = _hidden(rng, L, 20)
    y = near.astype(np.int32)
    y[[3, 9]] = -100
    dloss = np.ones(20, np.float32)
    good = _run(env, L, h, y, None, 1.0, dloss)
    h[3], h[9], dloss[9] = np.nan, np.inf, np.inf
    bad = _run(env, L, h, y, None, 1.0, dloss)
    keep = torch.tensor([t for t in range(20) if t not in (3, 9)], device="cuda")
    for a, b in zip(good, bad):
        assert torch.equal(a[keep], b[keep])
    assert not bad[0][[3, 9]].any() and not bad[3][[3, 9]].any()
    # a token that takes part with a NaN shows it, in its own row alone
    y[3] = 5
    worse = _run(env, L, h, y, None, 1.0, dloss)
    assert torch.isnan(worse[0][3]) and torch.isnan(worse[3][3]).all()
    for a, b in zip(good, worse):
        assert torch.equal(a[keep], b[keep])


def test_very_sure_and_very_spread_tokens(env):
    """Logits of hundreds: probabilities that are 1 and 0 to fp32."""
    L = Layer(env, 300, 256, 4, 128, 2)
    rng = np.random.default_rng(5)
    h, near = _hidden(rng, L, 24, sure=60.0)
    h[:4] = 0                                        # all entries alike
    for y in (near, (near + 1) % 300):
        g = np.ones(24, np.float32)
        _compare(env, L, h, y.astype(np.int32), None, 1.0, g, _run(env, L, h, y.astype(np.int32), None,
                                                                   1.0, g))


def test_gradients_are_the_losses_differences(env):
    """dh against central differences of the GPU's own losses along random
    directions d. The two losses are off by about 2^-20 of lse and the logits'
    sizes together, taken as 2^-17 (|loss| + 12); dh's elements by 2^-10 or
    so, far under 2% of |dh| |d| / sqrt(cols), the size of their product; the
    logits move by 0.01, so third derivatives count 1e-5."""
    torch, gq = env
    L = Layer(env, 400, 256, 4, 128, 3)
    rng = np.random.default_rng(6)
    m = 16
    h, near = _hidden(rng, L, m)
    index, logits = _teacher(rng, m, 8, 400, near)
    g = np.ones(m, np.float32)
    dh = _run(env, L, h, index, logits, 2.0, g)[3].cpu().numpy().astype(np.float64)
    for seed in range(4):
        d = np.random.default_rng(seed).choice([-1.0, 1.0], h.shape) * 2.0 ** -5
        up, down = (h.astype(np.float64) + d).astype(np.float16), (h.astype(np.float64) - d).astype(np.float16)
        lu, ld = (_run(env, L, v, index, logits, 2.0, g)[0].cpu().numpy().astype(np.float64)
                  for v in (up, down))
        real = (up.astype(np.float64) - down.astype(np.float64))
        want = (dh * real).sum(1)
        size = np.sqrt((dh ** 2).sum(1) * (real ** 2).sum(1)) / np.sqrt(h.shape[1])
        assert np.all(np.abs(lu - ld - want) <= 0.02 * size + 2.0 ** -17 * (np.abs(lu) + 12))


def test_any_stream_any_workspace_again_and_strided(env):
    torch, gq = env
    L = Layer(env, 700, 256, 4, 128, 4)
    rng = np.random.default_rng(7)
    m = 140
    h, near = _hidden(rng, L, m)
    i, t = (_cuda(env, a) for a in _teacher(rng, m, 8, 700, near))
    y, g = _cuda(env, _labels(rng, m, 700, near)), _cuda(env, rng.standard_normal(m), np.float32)
    wide = torch.full((m, 264), 9.0, dtype=torch.float16, device="cuda")
    wide[:, :256] = _cuda(env, h)
    hd = _cuda(env, h)
    need = max(gq.head_workspace_bytes(op, m, 700, 256, 8)
               for op in (gq.OP_HEAD_LOSS, gq.OP_HEAD_BACKWARD))

    def all_of(h, fill, stream, out=None):
        ws = None if fill is None else torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        k = dict(workspace=ws, stream=stream)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        a = gq.head_loss(h, *L.args, y, **k)
        da = gq.head_loss_backward(h, *L.args, y, a[1], a[2], g, out=out, **k)
        da = da.clone() if out is not None else da
        b = gq.head_distill(h, *L.args, i, t, 2.0, **k)
        db = gq.head_distill_backward(h, *L.args, i, t, 2.0, b[1], b[2], g, out=out, **k)
        torch.cuda.synchronize()
        return (*a, da, *b, db)

    first = all_of(hd, None, None)
    buf = torch.full((m + 2, 261), 7.0, dtype=torch.float16, device="cuda")
    for a in ((hd, 0, None), (hd, 255, None), (hd, 127, torch.cuda.Stream()), (wide[:, :256], None, None),
              (hd, None, None, buf[1:m + 1, 2:258])):
        for p, q in zip(first, all_of(*a)):
            assert torch.equal(p, q)
    buf[1:m + 1, 2:258] = 7.0
    assert bool((buf == 7.0).all())


def test_replayed_from_a_graph(env):
    torch, gq = env
    L = Layer(env, 700, 256, 4, 128, 4)
    rng = np.random.default_rng(8)
    m = 33
    h = torch.zeros((m, 256), dtype=torch.float16, device="cuda")
    y = torch.zeros((m,), dtype=torch.int32, device="cuda")
    g = torch.ones((m,), device="cuda")
    need = max(gq.head_workspace_bytes(op, m, 700, 256) for op in (gq.OP_HEAD_LOSS, gq.OP_HEAD_BACKWARD))
    new = lambda: dict(f=[torch.empty((m,), device="cuda") for _ in range(3)],  # noqa: E731
                       dh=torch.empty((m, 256), dtype=torch.float16, device="cuda"),
                       ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    o, e = new(), new()

    def step(o):
        gq.head_loss(h, *L.args, y, *o["f"], workspace=o["ws"])
        gq.head_loss_backward(h, *L.args, y, o["f"][1], o["f"][2], g, out=o["dh"], workspace=o["ws"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(o)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o)
    for rep in range(4):
        hn, near = _hidden(rng, L, m)
        h.copy_(_cuda(env, hn))
        y.copy_(_cuda(env, _labels(rng, m, 700, near)))
        torch.cuda.synchronize()
        graph.replay()
        step(e)
        torch.cuda.synchronize()
        for a, b in zip(o["f"] + [o["dh"]], e["f"] + [e["dh"]]):
            assert torch.equal(a, b), rep


def test_python_refusals(env):
    torch, gq = env
    L = Layer(env, 300, 256, 4, 128, 1)
    h = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    y = torch.zeros((4,), dtype=torch.int32, device="cuda")
    f = torch.zeros((4,), device="cuda")
    i, t = torch.zeros((4, 3), dtype=torch.int32, device="cuda"), torch.zeros((4, 3), device="cuda")
    for bad in (y.long(), y[:3], y.cpu(), i):
        with pytest.raises(ValueError):
            gq.head_loss(h, *L.args, bad)
    for bi, bt in ((i.long(), t), (i[:3], t), (i, t.half()), (i, t[:, :2]), (y, t), (i.cpu(), t)):
        with pytest.raises(ValueError):
            gq.head_distill(h, *L.args, bi, bt)
    for a in ((f[:3], f, f), (f, f.double(), f), (f, f, f.cpu())):
        with pytest.raises(ValueError):
            gq.head_loss_backward(h, *L.args, y, *a)
    with pytest.raises(ValueError):
        gq.head_distill_backward(h, *L.args, i, t, 1.0, f, f, f)  # student_logits is m x top
    with pytest.raises(ValueError):
        gq.head_loss(h, *L.args, y, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")[:16])
    with pytest.raises(gq.GPTQError, match="UNSUPPORTED"):
        gq.head_loss(torch.zeros((4, 260), dtype=torch.float16, device="cuda")[:, 2:258], *L.args, y)


# ------------------------------------------------------------ a run of them together
def _sixteen(a):
    return a.astype(np.float16).astype(np.float64)


def test_a_step_of_adapters_through_a_block_and_the_projection(env):
    """x -> up (adapters, ReLU) -> down (adapters) -> vocabulary loss and back
    to every adapter, then the decode product of the result. The oracle takes
    the same steps in fp64 and rounds where a tensor is handed on in fp16; an
    fp16 tensor may differ from its fp64 form by its rounding, 2^-11 (twice:
    two sides round), and carries that into what follows, so the gradients are
    compared by norm: five such hand-overs, each at most 2^-10 of the norm."""
    torch, gq = env
    rng = np.random.default_rng(11)
    m, d, f, vocab, n, r = 96, 256, 512, 700, 3, 8
    up, down, head = Layer(env, f, d, 4, 128, 1), Layer(env, d, f, 4, 128, 2), Layer(env, vocab, d, 8, 128, 3)
    x = (rng.standard_normal((m, d)) * 3).astype(np.float16)
    idx = (np.arange(m) // 40).astype(np.int32)
    a1, a2 = _adapters(rng, n, r, f, d), _adapters(rng, n, r, d, f)
    y = rng.integers(0, vocab, m).astype(np.int32)
    y[::9] = -100
    valid = y >= 0
    dloss = (valid * 1024.0 / valid.sum()).astype(np.float32)

    xd, i, t1, t2 = _cuda(env, x), _cuda(env, idx), [_cuda(env, a) for a in a1], [_cuda(env, a) for a in a2]
    h1 = gq.linear_forward_adapters(xd, *up.args, *t1, i, relu=True)
    h2 = gq.linear_forward_adapters(h1, *down.args, *t2, i)
    yd, gd = _cuda(env, y), _cuda(env, dloss)
    loss, lse, zk = gq.head_loss(h2, *head.args, yd)
    dh2 = gq.head_loss_backward(h2, *head.args, yd, lse, zk, gd)
    dh1, dA2, dB2 = gq.linear_backward_adapters(dh2, h1, *down.args, *t2, i)
    dpre = dh1 * (h1 > 0)
    dx, dA1, dB1 = gq.linear_backward_adapters(dpre, xd, *up.args, *t1, i)
    torch.cuda.synchronize()

    r1 = _sixteen(np.maximum(oracle.adapters_forward(x, up.W, *a1, idx), 0))
    r2 = _sixteen(oracle.adapters_forward(r1, down.W, *a2, idx))
    rl = oracle.head_loss(r2, head.W, y)[0]
    g2 = _sixteen(oracle.head_backward(r2, head.W, y, dloss))
    g1, rA2, rB2 = oracle.adapters_backward(g2, r1, down.W, *a2, idx)
    g1 = _sixteen(g1) * (r1 > 0)
    gx, rA1, rB1 = oracle.adapters_backward(g1, x, up.W, *a1, idx)
    near = lambda a, b: np.linalg.norm(a.cpu().numpy() - b) / np.linalg.norm(b)  # noqa: E731
    for got, want in ((h1, r1), (h2, r2), (loss, rl), (dh2, g2), (dA2, rA2), (dB2, rB2), (dpre, g1),
                      (dx, gx), (dA1, rA1), (dB1, rB1)):
        assert near(got, want) <= 5 * 2.0 ** -10

    # the decode product and the product for many tokens are the same layer
    y32 = gq.dequant_gemm_adapters(xd[:3].contiguous(), *up.args, *t1, i[:3].contiguous())
    both = torch.relu(y32).half().float() - h1[:3].float()
    assert both.abs().max() <= 2.0 ** -10 * h1[:3].abs().max()
