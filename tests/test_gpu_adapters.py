"""Low-rank adapters beside a stored layer, forward and backward, on the GPU
against the fp64 oracle, every output compared.

Bounds (u = 2^-24, one fp32 rounding; a sum of n products that are exact in
fp32 is off by at most n u times the sum of their sizes, in any order, and a
matrix instruction sums no less accurately than that):

  v = s A x     (cols + 2) u |s| sum |A x|: the products are exact, s once
  low = B v     v's error through |B|, and (rank + 2) u sum |B v|
  low (fp16)    in the products with fp16 outputs v is two fp16 numbers in units
                of the largest of 16 of its values: hi rounds to 2^-11, lo to
                half a step, 2^-25 or less of that unit where it is subnormal
                (2^-24 of the largest value, which is at least half a unit):
                2 u of it in all, through |B|; and the same sums as low
  y (decode)    the layer's own bound F u sum |x| (|q| + |z|) s (as for the
                product without adapters), low's, and one rounding of the sum
  y (fp16)      (cols + 2 ngroups + 2) u sum |x| |q - z| s (the sums of many
                tokens are kept in units of the current group's scale: two
                roundings a group), low's, 2 u |y|, and half an fp16 step at
                |y| plus all that
  dx            W_hat rounds to fp16 (2^-11 of it, or 2^-25 below 2^-14; 2 u for
                its fp32 form), (rows + 2) u sum |dy W|, A^T dv as low, half an
                fp16 step
  dA = dv^T x   dv's error (rows + 2) u, and the sum over the adapter's tokens,
                (tokens + chunks + 2) u; dB the same with v, (cols + 2) u
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    import post_weight_quantization_02_amd as gq
    return torch, gq


def _cuda(env, a, dtype=None):
    return env[0].from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def half_step16(v):
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -30))
    return np.ldexp(0.5, np.maximum(e - 1, -14) - 10)


class Layer:
    """A stored layer from the oracle's round-to-nearest codes."""

    def __init__(self, env, rows, cols, bits, g, seed, act_order=False):
        torch, gq = env
        r = oracle.rtn(np.random.default_rng(seed).standard_normal((rows, cols)) * 0.02, bits, g,
                       precision="f32")
        self.rows, self.cols, self.bits, self.g = rows, cols, bits, g
        self.codes = r["codes"]
        self.s = r["scales"].astype(np.float32).astype(np.float64)
        self.z = r["zeros"].astype(np.float32).astype(np.float64)
        gg = cols if g <= 0 or g > cols else g
        self.gg, self.ng = gg, -(-cols // gg)
        gi = np.arange(cols) // gg
        self.g_idx = None
        if act_order:
            perm = np.random.default_rng(seed + 1).permutation(cols)
            gi = np.empty(cols, np.int64)
            gi[perm] = np.arange(cols) // gg
            self.g_idx = _cuda(env, gi, np.int32)
        self.W = (self.codes - self.z[:, gi]) * self.s[:, gi]
        self.Wmag = (np.abs(self.codes) + np.abs(self.z[:, gi])) * self.s[:, gi]
        self.args = (_cuda(env, oracle.pack_codes(self.codes, bits).view(np.int32)), bits, cols,
                     _cuda(env, self.s, np.float32), _cuda(env, self.z, np.float32), g)


def _adapters(rng, n, rank, rows, cols):
    A = (rng.standard_normal((n, rank, cols)) / np.sqrt(cols)).astype(np.float16)
    B = (rng.standard_normal((n, rows, rank)) * 0.05).astype(np.float16)
    return A, B, (0.5 + rng.random(n)).astype(np.float32)


def _index(rng, kind, m, n):
    if kind == "mixed":
        return rng.integers(-1, n + 1, m).astype(np.int32)  # -1 and n: none
    if kind == "runs":
        return np.sort(rng.integers(0, n, m)).astype(np.int32)
    if kind == "none":
        return np.where(np.arange(m) % 2, -1, np.int32(2 ** 31 - 1)).astype(np.int32)
    return np.full(m, n - 1, np.int32)  # "last": one adapter for all


def _low(x, A, B, s, idx):
    """sum over |B| |s| |A| |x|: the adapters' part with every size positive."""
    return oracle.adapters_forward(np.abs(x.astype(np.float64)), np.zeros((B.shape[1], x.shape[1])),
                                   np.abs(A), np.abs(B), np.abs(s.astype(np.float64)), idx)


def _low_halves(x, A, B, s, idx):
    """2 u times each token's largest possible |v| through sum |B|."""
    out = np.zeros((len(x), B.shape[1]))
    for t, a in enumerate(oracle.adapter_of(idx, len(A))):
        if a >= 0:
            v = abs(float(s[a])) * (np.abs(A[a].astype(np.float64)) @ np.abs(x[t].astype(np.float64)))
            out[t] = 2 * U * v.max() * np.abs(B[a].astype(np.float64)).sum(1)
    return out


def _decode_bound(L, x, m):
    k = 32 // L.bits
    nw = -(-L.cols // k)
    f = max(max(-(-nw // 64) * k, 4 * k + -(-nw // 256)) + 8, 128 + -(-L.cols // 512) + 8)
    return f * U * (np.abs(x.astype(np.float64)) @ L.Wmag.T)


def _decode(env, L, m, n, rank, kind, seed, x=None):
    torch, gq = env
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, L.cols)).astype(np.float16) if x is None else x
    A, B, s = _adapters(rng, n, rank, L.rows, L.cols)
    idx = _index(rng, kind, m, n)
    y = gq.dequant_gemm_adapters(_cuda(env, x), *L.args, _cuda(env, A), _cuda(env, B), _cuda(env, s),
                                 _cuda(env, idx), g_idx=L.g_idx)
    torch.cuda.synchronize()
    ref = oracle.adapters_forward(x, L.W, A, B, s, idx)
    tol = _decode_bound(L, x, m) + (L.cols + rank + 6) * U * _low(x, A, B, s, idx) + U * np.abs(ref)
    err = np.abs(y.cpu().numpy() - ref)
    assert np.all(err <= tol), (float(err.max()), float(tol.min()))


@pytest.mark.parametrize("rows,cols,bits,g,m,n,rank,kind", [
    (1, 128, 4, 128, 1, 1, 1, "last"),          # the smallest
    (64, 256, 4, 128, 1, 2, 16, "last"),        # one token, x loaded directly
    (37, 384, 4, 128, 5, 3, 7, "mixed"),        # MFMA path, an odd rank
    (300, 1024, 4, 256, 33, 40, 16, "mixed"),   # two passes of the MFMA path
    (50, 1000, 3, 128, 5, 3, 8, "mixed"),       # words straddle groups, unaligned adapter rows
    (23, 77, 5, 16, 9, 2, 3, "mixed"),          # everything odd
    (40, 512, 2, 32, 2, 2, 64, "runs"),
    (9, 640, 8, 64, 4, 4, 128, "mixed"),        # the largest rank
    (50, 768, 4, 128, 70, 5, 33, "mixed"),      # beyond 64 tokens: 16-token tiles of v
    (30, 100, 4, 100, 90, 3, 20, "runs"),       # the same, scalar loads
    (40, 512, 4, 128, 3, 2, 16, "none"),        # no token has an adapter
    (45, 1280, 8, 256, 20, 4, 24, "mixed"),     # 8 bits, MFMA, 10 chunks over 8 waves
    (33, 256, 8, 0, 100, 3, 7, "runs"),         # the same, two passes of tokens
    (8200, 256, 4, 128, 20, 3, 16, "mixed"),    # 32 outputs a workgroup, the last one ragged
    (8195, 128, 8, 128, 3, 3, 8, "mixed"),
    (11, 9000, 6, 64, 3, 2, 8, "mixed"),        # more columns than fit the staging
    (11, 8300, 3, 16, 9, 2, 8, "mixed"),
])
def test_decode_with_adapters(env, rows, cols, bits, g, m, n, rank, kind):
    _decode(env, Layer(env, rows, cols, bits, g, rows + cols), m, n, rank, kind, seed=m + rank)


def test_decode_with_adapters_in_act_order(env):
    _decode(env, Layer(env, 40, 768, 4, 128, 5, act_order=True), 6, 3, 16, "mixed", seed=3)


@pytest.mark.parametrize("m", [1, 32])
def test_decode_full_layer_shape(env, m):
    _decode(env, Layer(env, 11008, 4096, 4, 128, 8), m, 16, 16, "mixed", seed=m)


def _forward(env, L, m, n, rank, kind, relu, seed):
    torch, gq = env
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, L.cols)).astype(np.float16)
    A, B, s = _adapters(rng, n, rank, L.rows, L.cols)
    idx = _index(rng, kind, m, n)
    y = gq.linear_forward_adapters(_cuda(env, x), *L.args, _cuda(env, A), _cuda(env, B),
                                   _cuda(env, s), _cuda(env, idx), relu=relu)
    torch.cuda.synchronize()
    ref = oracle.adapters_forward(x, L.W, A, B, s, idx)
    tol = (L.cols + 2 * L.ng + 2) * U * (np.abs(x.astype(np.float64)) @ np.abs(L.W).T) \
        + (L.cols + rank + 6) * U * _low(x, A, B, s, idx) + _low_halves(x, A, B, s, idx) \
        + 2 * U * np.abs(ref)
    tol += half_step16(np.abs(ref) + tol)
    if relu:
        ref = np.maximum(ref, 0)
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= tol), (float(err.max()), int((err > tol).sum()))


@pytest.mark.parametrize("m,rows,cols,bits,g,n,rank,kind,relu", [
    (1, 1, 128, 4, 128, 1, 1, "last", False),
    (129, 257, 256, 4, 128, 3, 16, "runs", True),     # one past a tile both ways
    (300, 600, 512, 4, 128, 5, 12, "mixed", False),   # every tile mixes adapters
    (200, 96, 384, 4, 0, 2, 128, "runs", False),      # per-channel, the largest rank
    (77, 300, 640, 8, 256, 3, 5, "mixed", True),
    (64, 130, 256, 8, 128, 2, 40, "runs", False),     # v by the kernel of few tokens
    (150, 256, 256, 4, 128, 2, 16, "none", False),
])
def test_forward_with_adapters(env, m, rows, cols, bits, g, n, rank, kind, relu):
    _forward(env, Layer(env, rows, cols, bits, g, m + rows), m, n, rank, kind, relu, seed=m + cols)


@pytest.mark.parametrize("cols,bits,g,n,rank,kind,relu", [
    (128, 4, 0, 2, 8, "runs", True),        # two stages, one group
    (640, 4, 256, 3, 20, "mixed", False),   # a short last group
    (384, 8, 128, 2, 16, "runs", False),    # three stages of 150 KB
    (640, 8, 256, 1, 5, "last", True),
])
def test_forward_in_the_largest_tiles(env, cols, bits, g, n, rank, kind, relu):
    """256 x 256, ragged both ways, with groups that add nothing: their scale
    is 0, in some rows all of them. The sums keep their unit through those."""
    L = Layer(env, 4200, cols, bits, g, cols + bits)
    L.s[::3, -1] = 0
    L.s[1::3, 0] = 0
    L.s[5::7] = 0
    gi = np.arange(cols) // L.gg
    L.W = (L.codes - L.z[:, gi]) * L.s[:, gi]
    L.Wmag = (np.abs(L.codes) + np.abs(L.z[:, gi])) * L.s[:, gi]
    L.args = (*L.args[:3], _cuda(env, L.s, np.float32), *L.args[4:])
    _forward(env, L, 2100, n, rank, kind, relu, seed=cols)


def test_tokens_without_adapter_get_the_layers_own_product(env):
    """Both products may add in another order than without adapters: each is
    within its own bound of the exact sum, the sum of the bounds apart, and
    the ones for many tokens are rounded to fp16 besides: a half step each,
    taken at the larger value."""
    torch, gq = env
    L = Layer(env, 96, 512, 4, 128, 1)
    rng = np.random.default_rng(2)
    for m, plain, with_ad in ((6, gq.dequant_gemm, gq.dequant_gemm_adapters),
                              (140, gq.linear_forward, gq.linear_forward_adapters)):
        x = _cuda(env, rng.standard_normal((m, 512)).astype(np.float16))
        A, B, s = (_cuda(env, a) for a in _adapters(rng, 2, 16, 96, 512))
        idx = torch.tensor([-1, 0] * (m // 2), dtype=torch.int32, device="cuda")
        y0, y = plain(x, *L.args), with_ad(x, *L.args, A, B, s, idx)
        y0, y, x = (v.cpu().numpy().astype(np.float64) for v in (y0, y, x))
        if m == 6:
            tol = 2 * _decode_bound(L, x, m)
        else:
            tol = (L.gg + L.cols + 3 * L.ng + 4) * U * (np.abs(x) @ np.abs(L.W).T)
            tol += 2 * half_step16(np.abs(y0) + tol)
        assert np.all(np.abs(y - y0)[0::2] <= tol[0::2])
        assert (y[1::2] != y0[1::2]).any()


def test_one_adapters_infinities_stay_with_its_tokens(env):
    torch, gq = env
    L = Layer(env, 64, 256, 4, 128, 1)
    rng = np.random.default_rng(3)
    A, B, s = _adapters(rng, 3, 16, 64, 256)
    bad_A, bad_B = A.copy(), B.copy()
    bad_A[1], bad_B[1] = np.nan, np.inf
    for m in (5, 150):
        x = rng.standard_normal((m, 256)).astype(np.float16)
        idx = rng.integers(0, 3, m).astype(np.int32)
        dy = rng.standard_normal((m, 64)).astype(np.float16)
        keep = torch.from_numpy(idx != 1).cuda()
        for call in (gq.dequant_gemm_adapters, gq.linear_forward_adapters):
            good, bad = (call(_cuda(env, x), *L.args, _cuda(env, a), _cuda(env, b), _cuda(env, s),
                              _cuda(env, idx)) for a, b in ((A, B), (bad_A, bad_B)))
            assert torch.equal(good[keep], bad[keep])
            assert not torch.isfinite(bad[~keep]).any()
        good, bad = (gq.linear_backward_adapters(_cuda(env, dy), _cuda(env, x), *L.args, _cuda(env, a),
                                                 _cuda(env, b), _cuda(env, s), _cuda(env, idx))
                     for a, b in ((A, B), (bad_A, bad_B)))
        assert torch.equal(good[0][keep], bad[0][keep])
        for g, b in zip(good[1:], bad[1:]):
            assert torch.equal(g[[0, 2]], b[[0, 2]])


def test_a_tokens_infinity_stays_in_its_row_and_its_adapters_gradient(env):
    torch, gq = env
    L = Layer(env, 64, 256, 4, 128, 1)
    rng = np.random.default_rng(4)
    m = 300
    x = rng.standard_normal((m, 256)).astype(np.float16)
    dy = rng.standard_normal((m, 64)).astype(np.float16)
    x[17], dy[40] = np.inf, np.nan
    idx = (np.arange(m) % 3).astype(np.int32)
    idx[17] = idx[40] = 2
    A, B, s = (_cuda(env, a) for a in _adapters(rng, 3, 16, 64, 256))
    y = gq.linear_forward_adapters(_cuda(env, x), *L.args, A, B, s, _cuda(env, idx))
    ok = torch.isfinite(y).all(1).cpu().numpy()
    assert not ok[17] and ok.sum() == m - 1
    dx, dA, dB = gq.linear_backward_adapters(_cuda(env, dy), _cuda(env, x), *L.args, A, B, s,
                                             _cuda(env, idx))
    ok = torch.isfinite(dx).all(1).cpu().numpy()
    assert not ok[40] and ok.sum() == m - 1
    for g in (dA, dB):
        assert torch.isfinite(g[:2]).all() and not torch.isfinite(g[2]).all()


def _backward(env, L, m, n, rank, kind, seed, dy_scale=0.05):
    torch, gq = env
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, L.cols)).astype(np.float16)
    dy = (rng.standard_normal((m, L.rows)) * dy_scale).astype(np.float16)
    W16 = np.abs(L.W) * (2.0 ** -11 + 2 * U) + 2.0 ** -25
    ady, ax = np.abs(dy.astype(np.float64)), np.abs(x.astype(np.float64))
    tol = ady @ (W16 + (L.rows + 2) * U * np.abs(L.W))
    if n == 0:
        dx = gq.linear_backward(_cuda(env, dy), *L.args, g_idx=L.g_idx)
        ref = dy.astype(np.float64) @ L.W
    else:
        A, B, s = _adapters(rng, n, rank, L.rows, L.cols)
        idx = _index(rng, kind, m, n)
        dx, dA, dB = gq.linear_backward_adapters(_cuda(env, dy), _cuda(env, x), *L.args, _cuda(env, A),
                                                 _cuda(env, B), _cuda(env, s), _cuda(env, idx),
                                                 g_idx=L.g_idx)
        ref, rA, rB = oracle.adapters_backward(dy, x, L.W, A, B, s, idx)
        low, mA, mB = oracle.adapters_backward(ady, ax, np.zeros_like(L.W), np.abs(A), np.abs(B), s,
                                               idx)
        tol += (L.rows + rank + 6) * U * low + 2 * U * np.abs(ref)
        tol += _low_halves(dy, B.transpose(0, 2, 1), A.transpose(0, 2, 1), s, idx)
        sums = m + m // 256 + 8
        for got, want, mag, inner in ((dA, rA, mA, L.rows), (dB, rB, mB, L.cols)):
            err = np.abs(got.cpu().numpy() - want)
            assert np.all(err <= (inner + sums) * U * mag), (inner, float(err.max()))
    torch.cuda.synchronize()
    tol += half_step16(np.abs(ref) + tol)
    err = np.abs(dx.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= tol), (float(err.max()), int((err > tol).sum()))


@pytest.mark.parametrize("m,rows,cols,bits,g,n,rank,kind", [
    (1, 1, 1, 4, 128, 1, 1, "last"),
    (1, 64, 128, 4, 128, 0, 0, ""),              # the layer alone
    (130, 129, 257, 4, 128, 0, 0, ""),           # one past a tile, rows copied to padded ones
    (16, 64, 128, 4, 128, 2, 16, "mixed"),
    (17, 70, 130, 3, 128, 3, 5, "mixed"),        # odd sizes: scalar loads everywhere
    (300, 192, 320, 4, 64, 3, 16, "runs"),       # group 64
    (530, 203, 264, 4, 128, 6, 24, "mixed"),     # tiles of many adapters; dy copied, wide loads of it
    (513, 256, 256, 8, 128, 2, 40, "runs"),      # three chunks of tokens an adapter
    (600, 64, 640, 5, 256, 2, 128, "mixed"),     # the largest rank
    (257, 1000, 96, 2, 16, 4, 12, "mixed"),
    (100, 128, 256, 4, 0, 2, 8, "none"),
])
def test_backward(env, m, rows, cols, bits, g, n, rank, kind):
    _backward(env, Layer(env, rows, cols, bits, g, m + rows), m, n, rank, kind, seed=m + cols)


def test_backward_in_act_order_and_with_small_gradients(env):
    _backward(env, Layer(env, 96, 256, 4, 64, 3, act_order=True), 40, 2, 8, "mixed", seed=1)
    _backward(env, Layer(env, 96, 256, 4, 64, 3), 40, 2, 8, "mixed", seed=1, dy_scale=1e-6)


@pytest.mark.parametrize("m,rows,cols", [(2100, 1024, 4096), (700, 4096, 2304)])
def test_backward_large_tiles(env, m, rows, cols):
    """256 x 256 tiles, ragged (144 of them: the smaller ones) and whole."""
    _backward(env, Layer(env, rows, cols, 4, 128, 2), m, 3, 16, "runs", seed=m)


@pytest.mark.parametrize("m,rows,cols,bits,g,n,rank,kind", [
    (1, 1, 128, 4, 128, 0, 0, ""),               # the smallest: one stage, one row of it
    (1, 129, 256, 8, 128, 0, 0, ""),             # an odd last pair of rows
    (64, 640, 384, 4, 128, 2, 16, "mixed"),      # whole 64-token tile, splits of the rows
    (65, 1003, 512, 8, 256, 0, 0, ""),           # one past it; groups over two tiles of columns
    (128, 512, 640, 8, 0, 3, 7, "mixed"),        # per-channel
    (129, 512, 16384, 4, 128, 0, 0, ""),         # two tiles of tokens, 256 workgroups, no split
    (256, 320, 8192, 8, 128, 2, 8, "runs"),      # the most tokens, two splits at most
    (160, 256, 11008, 4, 128, 0, 0, ""),         # idle CUs: from the transposed copy
    (257, 256, 128, 4, 128, 0, 0, ""),           # one past the most tokens
])
def test_backward_of_few_tokens(env, m, rows, cols, bits, g, n, rank, kind):
    """Straight from the packed words up to 256 tokens, and its neighbours."""
    _backward(env, Layer(env, rows, cols, bits, g, m + rows), m, n, rank, kind, seed=m + cols)


def test_backward_takes_any_zeros(env):
    """Zeros that are no integers (a layer from elsewhere): the packed words
    and the transposed copy make the same weights of them, so a token alone and
    the same token among 257 differ by the order of fp32 sums alone:
    2 * rows * 2^-24 * sum |dy W| (each side is within rows half steps of the
    exact sum) and one rounding to fp16 each."""
    torch, gq = env
    L = Layer(env, 256, 512, 4, 128, 9)
    packed, bits, cols, scales, zeros, groupsize = L.args
    zeros = zeros + 0.37
    rng = np.random.default_rng(9)
    dy = rng.standard_normal((257, 256)).astype(np.float16)
    few = gq.linear_backward(_cuda(env, dy[:3]), packed, bits, cols, scales, zeros, groupsize)
    many = gq.linear_backward(_cuda(env, dy), packed, bits, cols, scales, zeros, groupsize)[:3]
    eye = torch.eye(256, dtype=torch.float16, device="cuda")
    W = gq.linear_backward(torch.cat([eye, eye[:1]]), packed, bits, cols, scales, zeros,
                           groupsize)[:256].double().cpu().numpy()
    mag = np.abs(dy[:3].astype(np.float64)) @ np.abs(W)
    few, many = few.double().cpu().numpy(), many.double().cpu().numpy()
    assert np.all(np.abs(few - many) <= 2 * 256 * 2.0**-24 * mag + 2 * 2.0**-11 * np.abs(many) + 2.0**-24)
    exact = dy[:3].astype(np.float64) @ W  # of the weights rounded to fp16, as both use them
    assert np.all(np.abs(few - exact) <= 256 * 2.0**-24 * mag + 2.0**-11 * np.abs(exact) * 1.001 + 2.0**-25)


def test_gradients_without_tokens_are_zero(env):
    torch, gq = env
    L = Layer(env, 64, 128, 4, 128, 1)
    A, B, s = (_cuda(env, a) for a in _adapters(np.random.default_rng(1), 2, 8, 64, 128))
    z = lambda c: torch.empty((0, c), dtype=torch.float16, device="cuda")  # noqa: E731
    idx = torch.empty((0,), dtype=torch.int32, device="cuda")
    nan = lambda t: torch.full(t.shape, float("nan"), device="cuda")  # noqa: E731
    dx, dA, dB = gq.linear_backward_adapters(z(64), z(128), *L.args, A, B, s, idx, dA=nan(A), dB=nan(B))
    assert dx.shape == (0, 128) and not dA.any() and not dB.any()
    assert gq.dequant_gemm_adapters(z(128), *L.args, A, B, s, idx).shape == (0, 64)
    assert gq.linear_forward_adapters(z(128), *L.args, A, B, s, idx).shape == (0, 64)


def test_strided_operands_and_untouched_surroundings(env):
    torch, gq = env
    L = Layer(env, 128, 256, 4, 128, 1)
    rng = np.random.default_rng(6)
    m = 150
    A, B, s = (_cuda(env, a) for a in _adapters(rng, 2, 16, 128, 256))
    idx = _cuda(env, _index(rng, "mixed", m, 2))
    wide = lambda w, pad: _cuda(env, rng.standard_normal((m, w + pad)).astype(np.float16))  # noqa: E731
    xw, dyw = wide(256, 8), wide(128, 24)
    x, dy = xw[:, :256], dyw[:, :128]
    buf = lambda w, dt: torch.full((m + 2, w + 5), 7.0, dtype=dt, device="cuda")  # noqa: E731

    def inside(b, w, got, want):
        assert torch.equal(got, want)
        rest = b.clone()
        rest[1:m + 1, 2:2 + w] = 7.0
        assert bool((rest == 7.0).all())

    for call, dt in ((gq.dequant_gemm_adapters, torch.float32),
                     (gq.linear_forward_adapters, torch.float16)):
        b = buf(128, dt)
        out = call(x, *L.args, A, B, s, idx, out=b[1:m + 1, 2:130])
        inside(b, 128, out, call(x.contiguous(), *L.args, A, B, s, idx))
    b = buf(256, torch.float16)
    out = gq.linear_backward_adapters(dy, x, *L.args, A, B, s, idx, out=b[1:m + 1, 2:258])
    want = gq.linear_backward_adapters(dy.contiguous(), x.contiguous(), *L.args, A, B, s, idx)
    inside(b, 256, out[0], want[0])
    assert torch.equal(out[1], want[1]) and torch.equal(out[2], want[2])


def test_same_results_in_any_stream_with_any_workspace_and_again(env):
    torch, gq = env
    L = Layer(env, 192, 256, 4, 128, 1)
    rng = np.random.default_rng(7)
    m = 300
    x = _cuda(env, rng.standard_normal((m, 256)).astype(np.float16))
    dy = _cuda(env, rng.standard_normal((m, 192)).astype(np.float16))
    A, B, s = (_cuda(env, a) for a in _adapters(rng, 4, 16, 192, 256))
    idx = _cuda(env, _index(rng, "mixed", m, 4))
    nf = gq.adapters_workspace_bytes(gq.OP_FORWARD_ADAPTERS, m, 192, 256, 4, 16)
    nb = gq.adapters_workspace_bytes(gq.OP_BACKWARD, m, 192, 256, 4, 16)

    def all_of(fill, stream):
        ws = None if fill is None else torch.full((max(nf, nb),), fill, dtype=torch.uint8, device="cuda")
        k = dict(workspace=ws, stream=stream)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        y = gq.dequant_gemm_adapters(x, *L.args, A, B, s, idx, **k)
        f = gq.linear_forward_adapters(x, *L.args, A, B, s, idx, **k)
        g = gq.linear_backward_adapters(dy, x, *L.args, A, B, s, idx, **k)
        torch.cuda.synchronize()
        return (y, f, *g)

    first = all_of(None, None)
    for fill, stream in ((0, None), (255, None), (127, torch.cuda.Stream()), (None, torch.cuda.Stream())):
        for a, b in zip(first, all_of(fill, stream)):
            assert torch.equal(a, b)


def test_memory_for_another_stream_is_not_taken_from_queued_work(env):
    """A tensor whose copy is still queued on the current stream is freed, and
    calls on another stream, which does not wait for it, allocate outputs and
    workspaces of its size: the copy still gets its values."""
    torch, gq = env
    L = Layer(env, 192, 256, 4, 128, 1)
    m = 300
    rng = np.random.default_rng(3)
    x = _cuda(env, rng.standard_normal((m, 256)).astype(np.float16))
    A, B, s = (_cuda(env, a) for a in _adapters(rng, 4, 16, 192, 256))
    idx = _cuda(env, _index(rng, "mixed", m, 4))
    want = gq.linear_forward_adapters(x, *L.args, A, B, s, idx)
    sizes = [gq.adapters_workspace_bytes(gq.OP_FORWARD_ADAPTERS, m, 192, 256, 4, 16), m * 192 * 2]
    busy = torch.zeros((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    olds = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    for _ in range(20):
        busy = busy @ busy
    copies = [o.clone() for o in olds]
    del olds
    got = gq.linear_forward_adapters(x, *L.args, A, B, s, idx, stream=side)
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    assert torch.equal(got, want)


def test_decode_and_training_step_replayed_from_a_graph(env):
    """Replays with inputs changed in between, other eager work on the same
    library between them, equal the eager results bit for bit."""
    torch, gq = env
    L = Layer(env, 192, 256, 4, 128, 1)
    rng = np.random.default_rng(8)
    m = 40
    x, dy = (torch.zeros((m, w), dtype=torch.float16, device="cuda") for w in (256, 192))
    A, B, s = (_cuda(env, a) for a in _adapters(rng, 4, 16, 192, 256))
    idx = torch.zeros((m,), dtype=torch.int32, device="cuda")
    size = max(gq.adapters_workspace_bytes(op, m, 192, 256, 4, 16)
               for op in (gq.OP_FORWARD_ADAPTERS, gq.OP_BACKWARD))
    new = lambda: dict(y=torch.empty((m, 192), device="cuda"),  # noqa: E731
                       dx=torch.empty((m, 256), dtype=torch.float16, device="cuda"),
                       dA=torch.empty(A.shape, device="cuda"), dB=torch.empty(B.shape, device="cuda"),
                       ws=torch.empty(size, dtype=torch.uint8, device="cuda"))
    o, e = new(), new()

    def step(o):
        gq.dequant_gemm_adapters(x, *L.args, A, B, s, idx, out=o["y"], workspace=o["ws"])
        gq.linear_backward_adapters(dy, x, *L.args, A, B, s, idx, out=o["dx"], dA=o["dA"], dB=o["dB"],
                                    workspace=o["ws"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(o)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(o)
    for rep in range(4):
        x.copy_(_cuda(env, rng.standard_normal((m, 256)).astype(np.float16)))
        dy.copy_(_cuda(env, rng.standard_normal((m, 192)).astype(np.float16)))
        idx.copy_(_cuda(env, _index(rng, ("mixed", "runs", "none", "last")[rep], m, 4)))
        torch.cuda.synchronize()
        g.replay()
        step(e)
        torch.cuda.synchronize()
        for k in ("y", "dx", "dA", "dB"):
            assert torch.equal(o[k], e[k]), (rep, k)


def test_python_refusals(env):
    torch, gq = env
    L = Layer(env, 64, 256, 4, 128, 1)
    rng = np.random.default_rng(9)
    x = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    dy = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    A, B, s = (_cuda(env, a) for a in _adapters(rng, 2, 16, 64, 256))
    idx = torch.zeros((4,), dtype=torch.int32, device="cuda")
    bad = [(A[:, :8], B, s, idx), (A.float(), B, s, idx), (A.cpu(), B, s, idx), (A, B[:, :63], s, idx),
           (A, B, s.double(), idx), (A, B, s[:1], idx), (A, B, s, idx.long()), (A, B, s, idx[:3]),
           (A.transpose(1, 2), B, s, idx), (A[0], B, s, idx), (A, B, s, idx.cpu())]
    for ad in bad:
        for call in (gq.dequant_gemm_adapters, gq.linear_forward_adapters):
            with pytest.raises(ValueError):
                call(x, *L.args, *ad)
        with pytest.raises(ValueError):
            gq.linear_backward_adapters(dy, x, *L.args, *ad)
    for badx in (x[:3], x.float(), x.cpu(), x[:, :128]):
        with pytest.raises(ValueError):
            gq.linear_backward_adapters(dy, badx, *L.args, A, B, s, idx)
    with pytest.raises(ValueError):
        gq.linear_backward_adapters(dy, x, *L.args, A, B, s, idx, dA=torch.empty_like(A))
    with pytest.raises(ValueError):
        gq.dequant_gemm_adapters(x, *L.args, A, B, s, idx,
                                 workspace=torch.empty(255, dtype=torch.uint8, device="cuda"))
    big = torch.zeros((2, 130, 256), dtype=torch.float16, device="cuda")
    with pytest.raises(gq.GPTQError, match="UNSUPPORTED"):
        gq.dequant_gemm_adapters(x, *L.args, big, torch.zeros((2, 64, 130), dtype=torch.float16,
                                                               device="cuda"), s, idx)
