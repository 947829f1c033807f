"""Per-head norm and rotation on the GPU against the oracle in 64 bits.

The bound, per element: the half step of the output type (2^-8 for bf16,
2^-24 for fp32) plus fp32 roundings of 2^-24 relative to |h_a| + |h_b|: the
sum of squares D/8/lanes + 8 + 5 additions (halved by the square root), the
division, eps, reciprocal root (2) and last product 4, the weight's sum 1, the
sine and cosine 2 plus the angle's rounding 1, products and the fused sum 3 --
below 24 + D / 16 together."""
import numpy as np
import pytest

import oracle
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


def frequencies(half, base=10000.0):
    return (base ** (-np.arange(half) / max(half, 1))).astype(np.float32)


def check(got, x, D, w, off, eps, pos, f, inter, dt, what=""):
    ref = oracle.qk_norm_rope(x, D, w, off, eps, pos, f, inter)
    h = np.abs(oracle.qk_norm_rope(x, D, w, off, eps, pos, None, inter)).reshape(x.shape[0], -1, D)
    half = 0 if f is None else len(f)
    mag = h.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        mag[:, :, a] = mag[:, :, b] = h[:, :, a] + h[:, :, b]
    tol = (2.0 ** -8 if dt == "bf16" else 2.0 ** -24) * np.abs(ref) + \
        (24 + D / 16) * 2.0 ** -24 * mag.reshape(ref.shape) + 1e-40
    bad = np.abs(got - ref) - tol
    assert np.isfinite(got).all() and bad.max() <= 0, f"{what}: {bad.max():.3e} beyond the bound at {np.unravel_index(bad.argmax(), bad.shape)}"


def draw(rng, M, heads, D, dt):
    x = rng.standard_normal((M, heads * D)) * np.exp(rng.standard_normal((M, 1)))
    return oracle.round_to(x, dt).astype(np.float32)


CASES = [  # M, hq, hk, D, rotary, start, interleaved, fused
    (1, 1, 1, 8, 8, 0, False, False), (1, 4, 1, 256, 256, 31000, False, False), (2, 3, 1, 64, 64, 5, True, False),
    (3, 5, 2, 80, 36, 1000000, True, True), (3, 5, 2, 80, 36, 1000000, False, True), (17, 6, 3, 96, 96, 7, False, False),
    (33, 2, 2, 128, 64, 100, False, True), (9, 7, 1, 128, 2, 9, False, False), (5, 3, 1, 192, 190, 3, False, False),
    (400, 2, 1, 72, 40, 3, False, True), (6, 2, 1, 512, 512, 8000, False, False), (4, 2, 2, 512, 128, 8000, True, True),
    (3, 1, 1, 1024, 1024, 77, False, False), (3, 1, 2, 1000, 500, 77, False, False), (7, 40, 8, 128, 128, 2, False, False),
    (600, 9, 3, 256, 256, 1, False, True), (5, 300, 2, 16, 16, 1, True, False), (4, 2, 1, 264, 264, 4, False, False),
    (5, 2, 0, 256, 0, 0, False, False)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("M,hq,hk,D,rotary,start,inter,fused", CASES)
def test_matches_oracle(lib, torch, M, hq, hk, D, rotary, start, inter, fused, in_place, dt):
    rng = np.random.default_rng(M + 10 * hq + hk + D + rotary)
    q, k = draw(rng, M, hq, D, dt), draw(rng, M, hk, D, dt)
    wq, wk = (oracle.round_to(0.1 * rng.standard_normal(D), dt).astype(np.float32) for _ in range(2))
    f = frequencies(rotary // 2) if rotary else None
    pos = start + rng.integers(0, 5, M).cumsum()
    # rows of a wider buffer with guard columns between and behind them
    pad = 8 if fused else 0
    buf = torch.full((M, (hq + hk) * D + 2 * pad), 7.0, dtype=dev(q, dt).dtype, device="cuda")
    nq = hq * D
    cut = (lambda t: (t[:, :nq], t[:, nq + pad:nq + pad + hk * D])) if fused else \
        (lambda t: (t[:, :nq].contiguous(), t[:, nq:].contiguous()))
    Q, K = cut(buf)
    Q.copy_(dev(q, dt))
    K.copy_(dev(k, dt))
    out = torch.full_like(buf, 7.0)
    Qo, Ko = (Q, K) if in_place else cut(out)
    if not hk:
        K = Ko = None
    lib.theta_qk_norm_rope(Q, K, dev(wq, dt), dev(wk, dt), torch.from_numpy(pos).cuda(),
                           None if f is None else torch.from_numpy(f).cuda(), Qo, Ko, D, eps=1e-6, weight_offset=1.0,
                           interleaved=inter)
    lib.theta_device_status()
    check(host(Qo), q, D, wq, 1.0, 1e-6, pos, f, inter, dt, "q")
    if hk:
        check(host(Ko), k, D, wk, 1.0, 1e-6, pos, f, inter, dt, "k")
    if fused:
        for t in (buf, out):
            assert (t[:, nq:nq + pad] == 7).all() and (t[:, nq + pad + hk * D:] == 7).all()
    if not in_place:
        assert np.array_equal(host(Q), q)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_without_weights_and_positions(lib, torch, dt):
    """The norm alone, as some models apply it to the values."""
    rng = np.random.default_rng(1)
    x = draw(rng, 5, 3, 128, dt)
    X = dev(x, dt)
    Y = torch.empty_like(X)
    lib.theta_qk_norm_rope(X, None, None, None, None, None, Y, None, 128, eps=1e-5, weight_offset=1.0)
    lib.theta_device_status()
    check(host(Y), x, 128, None, 0.0, 1e-5, None, None, False, dt)


@pytest.mark.parametrize("pos", [[0, -1, -77777], [2 ** 31 - 1, 2 ** 31, 16777217], [1048576, 131071, 999999]])
def test_far_positions(lib, torch, pos):
    """Positions beyond fp32's whole numbers and below zero: angles are formed in fp64."""
    rng = np.random.default_rng(2)
    x = draw(rng, 3, 2, 64, "f32")
    p = np.array(pos, np.int64)
    f = frequencies(32)
    X, Y = dev(x), torch.empty(3, 128, device="cuda")
    lib.theta_qk_norm_rope(X, None, None, None, torch.from_numpy(p).cuda(), torch.from_numpy(f).cuda(), Y, None, 64)
    lib.theta_device_status()
    # the oracle's own fp64 angles, numpy's reduction of large arguments
    got, ref = host(Y), oracle.qk_norm_rope(x, 64, None, 0.0, 1e-6, p, f, False)
    tol = 2.0 ** -24 * np.abs(ref) + (28 * 2.0 ** -24 + (2.0 ** -19 if max(pos) > 2 ** 30 else 0)) * 2 * np.abs(x).max()
    assert np.all(np.abs(got - ref) <= tol * 2)


def test_zero_heads_huge_heads_and_bad_values(lib, torch):
    """A head of zeros stays zero (eps), a head with a NaN or an infinity is
    NaN as the formula gives, its neighbours are untouched by it."""
    rng = np.random.default_rng(4)
    x = draw(rng, 3, 4, 64, "f32")
    x[1, :64] = 0.0
    x[1, 64 + 10] = np.nan
    x[2, 128 + 3] = np.inf
    X, Y = dev(x), torch.empty(3, 256, device="cuda")
    f = frequencies(16)
    pos = np.array([1, 2, 3])
    lib.theta_qk_norm_rope(X, None, None, None, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), Y, None, 64)
    lib.theta_device_status()
    y = host(Y)
    assert not y[1, :64].any() and np.isnan(y[1, 64:128]).all()
    # the infinity's head: r = 0, so finite values become 0 and it (and its pair) NaN
    h = y[2, 128:192]
    assert np.isnan(h[[3, 19]]).all() and not np.delete(h, [3, 19]).any()
    clean = np.ones((3, 4), bool)
    clean[1, 1] = clean[2, 2] = False
    xs, ys = x.reshape(3, 4, 64), y.reshape(3, 4, 64)
    for m, hh in zip(*np.nonzero(clean)):
        check(ys[m, hh][None], xs[m, hh][None], 64, None, 0.0, 1e-6, pos[m:m + 1], f, False, "f32")


def test_past_32_bit_offsets_in_place(lib, torch):
    """A query buffer of more than 2^31 elements, in place, many rounds of tokens a block."""
    M, heads, D = 300000, 30, 256
    rng = np.random.default_rng(6)
    x = draw(rng, 8, heads, D, "bf16")
    X = dev(x, "bf16").repeat(M // 8, 1)
    f = frequencies(D // 2)
    pos = torch.arange(M, device="cuda")
    lib.theta_qk_norm_rope(X, None, None, None, pos, torch.from_numpy(f).cuda(), X, None, D)
    lib.theta_device_status()
    for at in (0, M // 2, M - 8):
        check(host(X[at:at + 8]), x, D, None, 0.0, 1e-6, np.arange(at, at + 8), f, False, "bf16", f"token {at}")


def test_captured_other_stream_and_side_by_side(lib, torch):
    rng = np.random.default_rng(5)
    x = draw(rng, 40, 6, 128, "bf16")
    f = torch.from_numpy(frequencies(64)).cuda()
    pos = torch.arange(40, device="cuda")
    X, Y = dev(x, "bf16"), torch.empty(40, 768, dtype=torch.bfloat16, device="cuda")
    args = (X[:, :512], X[:, 512:], None, None, pos, f, Y[:, :512], Y[:, 512:], 128)
    lib.theta_qk_norm_rope(*args)
    want = Y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y.zero_()
    torch.cuda.synchronize()
    lib.theta_qk_norm_rope(*args, stream=side)
    side.synchronize()
    assert torch.equal(Y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.theta_qk_norm_rope(*args)
    Y.zero_()
    g.replay()
    lib.theta_device_status()
    assert torch.equal(Y, want)


def test_binding_refusals_on_the_gpu(lib, torch):
    X = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    f, pos = torch.ones(32, device="cuda"), torch.arange(4, device="cuda")
    ok = dict(Q=X, K=None, q_weight=None, k_weight=None, positions=pos, inv_freq=f, Q_out=X, K_out=None, head_dim=64)
    for bad in (dict(head_dim=60), dict(head_dim=0), dict(positions=pos.int()), dict(positions=pos[:2]),
                dict(inv_freq=f.double()), dict(Q_out=X.float()), dict(Q_out=X[:, :128]), dict(K=X), dict(K_out=X),
                dict(q_weight=torch.zeros(64, device="cuda")), dict(q_weight=X[0, :32]), dict(Q=X.t()),
                dict(Q=X[:, ::2]), dict(positions=pos.cpu())):
        with pytest.raises((ValueError, TypeError)):
            lib.theta_qk_norm_rope(**{**ok, **bad})
    for bad in (dict(positions=None), dict(inv_freq=torch.ones(33, device="cuda"))):
        with pytest.raises(lib.ThetaError):
            lib.theta_qk_norm_rope(**{**ok, **bad})
