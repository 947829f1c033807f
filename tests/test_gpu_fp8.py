"""Block-scaled FP8 on the GPU: both encoders bit for bit against the oracle
(blocks over many decades, zero blocks, subnormals, values that are not
finite, ragged edges), the forward against the oracle's 64-bit forward of the
same codes over every range of token counts, and the run of them together.

The forward's bound, per element, with A the sum of the terms' magnitudes:
the products of two E4M3 values are exact and so are the power-of-two scales;
the tensor cores add 32 (FP8) or 16 (bf16) products at a time into an fp32
accumulator, each addition off by at most 2^-22 of the magnitudes summed so far
(the addends are aligned to the largest and cut), and split sums, s and the
last addition add fewer than 24 roundings of 2^-24: (I / 32 + 8) 2^-22 A for
the main term. T = X.V is held to 2^-16 (a high and a low bf16 part) on top of
its own sum: ((I + r) / 16 + 8) 2^-22 + 2^-16 of the rank term's magnitudes.
One rounding to bf16 is 2^-8 of the value (half a step), of at least the
smallest normal number."""
import numpy as np
import pytest

import oracle
import synthetic as syn
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


def encode(lib, torch, W):
    O, I = W.shape
    c = torch.full((O, I), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-O // 128), -(-I // 128)), 0xAA, dtype=torch.uint8, device="cuda")
    lib.theta_fp8_quantize(W, c, s)
    return c, s


def encode_rows(lib, torch, X):
    M, I = X.shape
    c = torch.full((M, I), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-I // 128), M), 0xAA, dtype=torch.uint8, device="cuda")
    lib.theta_fp8_quantize_rows(X, c, s)
    return c, s


def varied(rows, cols, seed, dt):
    """Values over many decades: per row and per 128 columns another size; a
    zero block, tiny and subnormal blocks, exact ties, values not finite."""
    rng = np.random.default_rng(seed)
    W = rng.standard_normal((rows, cols)) * 10.0 ** rng.uniform(-3, 3, (rows, 1))
    W *= np.repeat(10.0 ** rng.uniform(-8, 8, -(-cols // 128)), 128)[:cols]
    W[0, :16] = [448, -448, 0.0, -0.0, 1.0625, 1.1875, -1.0625, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17, 19, 240, 249,
                 1e-30, -1e-30]
    if cols > 128:
        W[:, 128:144] *= 1e-36
        if rows > 130:
            W[128:, 128:256] = 0.0
    if rows > 2:
        W[1, 3], W[2, 5], W[2, 6] = np.inf, -np.inf, np.nan
    return oracle.round_to(W, dt).astype(np.float32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("O,I", [(1, 16), (8, 128), (128, 256), (129, 144), (300, 1168), (257, 4096)])
def test_quantize_is_bit_exact(lib, torch, O, I, dt):
    W = varied(O, I, O + I, dt)
    c, s = encode(lib, torch, dev(W, dt))
    cr, sr = oracle.fp8_quantize(W)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(c.cpu().numpy(), cr)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,I", [(1, 16), (1, 5376), (2, 640), (17, 144), (63, 1168), (130, 2064)])
def test_quantize_rows_is_bit_exact(lib, torch, M, I, dt):
    X = varied(M, I, M + I, dt)
    c, s = encode_rows(lib, torch, dev(X, dt))
    cr, sr = oracle.fp8_quantize_rows(X)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(c.cpu().numpy(), cr)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_signs_and_infinities_at_block_edges(lib, torch, dt):
    """Every NaN and infinity, either sign, gets the code 0x7f; the block's
    other values keep the scale of its finite ones."""
    rng = np.random.default_rng(9)
    W = oracle.round_to(rng.standard_normal((160, 272)), dt).astype(np.float32)
    t = dev(W, dt)
    bits = t.view(torch.int16 if dt == "bf16" else torch.int32)
    for (r, c), b in (((0, 0), 0x7F81), ((127, 127), 0xFFC0), ((128, 128), 0xFF80), ((159, 271), 0x7F80),
                      ((5, 255), 0xFFFF)):
        b = b if dt == "bf16" else b << 16
        bits[r, c] = b - (1 << 16 if dt == "bf16" else 1 << 32) if b >> (15 if dt == "bf16" else 31) else b
        W[r, c] = np.nan
    for enc, ref in ((encode, oracle.fp8_quantize), (encode_rows, oracle.fp8_quantize_rows)):
        c, s = enc(lib, torch, t)
        cr, sr = ref(W)
        assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(c.cpu().numpy(), cr)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scale_extremes(lib, torch, dt):
    """Blocks whose largest value is at either end of the type's range, or just
    at and just above 448 times a power of two."""
    rows = np.zeros((6, 128), np.float64)
    big = float(torch.finfo(torch.bfloat16 if dt == "bf16" else torch.float32).max)
    tiny = 2.0 ** -133 if dt == "bf16" else 2.0 ** -149
    for m, a in enumerate([big, tiny, 448.0 * 2.0 ** 20, 450.0 * 2.0 ** 20, 2.0 ** -126, 1.75 * 2.0 ** -118]):
        rows[m, 5], rows[m, 6] = a, -a / 2
    X = oracle.round_to(rows, dt).astype(np.float32)
    c, s = encode_rows(lib, torch, dev(X, dt))
    cr, sr = oracle.fp8_quantize_rows(X)
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(c.cpu().numpy(), cr)


# ------------------------------------------------------------------ forward
class Problem:
    def __init__(self, lib, torch, M, O, I, r, seed=None, x_rows=1.0):
        seed = M + O + I + r if seed is None else seed
        self.lib, self.torch, self.dims = lib, torch, (M, O, I, r)
        rng = np.random.default_rng(seed)
        X = rng.standard_normal((M, I)) * np.exp(rng.standard_normal((M, 1))) * x_rows
        self.X = oracle.round_to(X, "bf16").astype(np.float32)
        W = syn.host_normal((O, I), 0.02, seed, "W0", O, I, dtype="bf16")
        self.s = (1.0 + syn.host_normal((O,), 0.05, seed, "s", O)).astype(np.float32)
        self.U = syn.host_normal((O, r), 0.05, seed, "U", O, r, dtype="bf16")
        self.V = syn.host_normal((I, r), 0.05, seed, "V", I, r, dtype="bf16")
        self.Xd, self.sd = dev(self.X, "bf16"), dev(self.s)
        self.Ud, self.Vd = (dev(self.U, "bf16"), dev(self.V, "bf16")) if r else (None, None)
        self.xc, self.xs = encode_rows(lib, torch, self.Xd)
        self.wc, self.ws = encode(lib, torch, dev(W, "bf16"))
        nb = lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, M, O, I, r, lib.THETA_BF16)
        self.work = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        self.guard = torch.full((M * O + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.Y = self.guard[256:256 + M * O].view(M, O)

    def call(self, **kw):
        self.lib.theta_linear_forward_fp8(self.Xd if self.dims[3] else None, self.xc, self.xs, self.wc, self.ws,
                                          self.sd, self.Ud, self.Vd, self.Y, self.work if self.dims[3] else None, **kw)
        return self.Y

    def values(self, rows=slice(None)):
        x = oracle.fp8_dequantize_rows(self.xc.cpu().numpy(), self.xs.cpu().numpy())
        w = oracle.fp8_dequantize(self.wc.cpu().numpy(), self.ws.cpu().numpy())[rows]
        return x, w

    def check(self, Y=None, rows=slice(None), what=""):
        M, O, I, r = self.dims
        Y = host(self.Y if Y is None else Y)[:, rows]
        x, w = self.values(rows)
        s = self.s.astype(np.float64)[rows]
        ref, A = (x @ w.T) * s, (np.abs(x) @ np.abs(w).T) * np.abs(s)
        tol = (I / 32 + 8) * 2.0 ** -22 * A
        if r:
            X, U, V = (a.astype(np.float64) for a in (self.X, self.U[rows], self.V))
            ref = ref + (X @ V) @ U.T
            tol = tol + (((I + r) / 16 + 8) * 2.0 ** -22 + 2.0 ** -16) * ((np.abs(X) @ np.abs(V)) @ np.abs(U).T)
        tol = tol + 2.0 ** -8 * np.maximum(np.abs(ref) + tol, 2.0 ** -126)
        bad = np.abs(Y - ref) - tol
        assert np.isfinite(Y).all() and bad.max() <= 0, f"{what}: off by {bad.max():.3e} beyond the bound at {np.unravel_index(bad.argmax(), bad.shape)}"
        assert (self.guard[:256] == 7).all() and (self.guard[256 + M * O:] == 7).all(), "wrote outside Y"


SHAPES = [(1, 8, 16, 0), (1, 256, 1152, 32), (1, 1032, 640, 8), (2, 392, 336, 24), (2, 264, 400, 256), (1, 136, 16, 200), (1, 264, 256, 256), (2, 264, 272, 240), (1, 520, 8192, 8),
          (2, 520, 8208, 8), (2, 136, 1648, 40), (3, 136, 144, 16), (1, 6912, 1152, 0),
          (5, 128, 128, 8), (8, 264, 4096, 64), (15, 1024, 1152, 40), (16, 2048, 5376, 64), (17, 128, 2064, 0),
          (31, 520, 1296, 256), (33, 776, 272, 32), (64, 1152, 6912, 32), (65, 136, 512, 128), (100, 1000, 1168, 24),
          (128, 256, 1152, 0), (129, 384, 256, 8), (200, 2056, 1168, 24), (256, 1024, 1152, 64), (257, 264, 656, 16),
          (333, 2056, 1168, 24), (520, 1288, 400, 72), (777, 4104, 272, 0), (1000, 520, 2064, 200)]


@pytest.mark.parametrize("policy", ["latency", "throughput"])
@pytest.mark.parametrize("M,O,I,r", SHAPES)
def test_forward_matches_oracle(lib, torch, M, O, I, r, policy):
    p = Problem(lib, torch, M, O, I, r)
    lib.theta_set_policy(lib.THETA_POLICY_THROUGHPUT if policy == "throughput" else lib.THETA_POLICY_LATENCY)
    try:
        p.call()
        lib.theta_device_status()
    finally:
        lib.theta_set_policy(lib.THETA_POLICY_LATENCY)
    p.check(what=f"{M}x{O}x{I} r{r} {policy}")


@pytest.mark.parametrize("M", [1, 2, 16, 300])
def test_same_result_twice(lib, torch, M):
    p = Problem(lib, torch, M, 1160, 1296, 32)
    a = p.call().clone()
    p.work.fill_(0xFF)
    assert torch.equal(a, p.call())
    lib.theta_device_status()


@pytest.mark.parametrize("M", [1, 2, 40, 300])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e25])
def test_far_scales(lib, torch, M, size):
    """Tokens far from unit size, next to ordinary ones in one call."""
    rows = np.ones((M, 1))
    rows[0] = size
    p = Problem(lib, torch, M, 520, 656, 16, x_rows=rows)
    p.call()
    lib.theta_device_status()
    p.check(what=f"size {size}")


@pytest.mark.parametrize("M", [1, 2, 7, 64, 300])
def test_values_not_finite_stay_in_their_rows(lib, torch, M):
    """A NaN or infinity in a token makes that token's outputs NaN, one in W0
    its column, and leaves the others as they are."""
    O, I = 264, 400
    p = Problem(lib, torch, M, O, I, 0)
    clean = host(p.call())
    p.xc[M // 2, 130] = 0x7F
    p.wc[200, 399] = 0xFF
    y = host(p.call())
    lib.theta_device_status()
    bad = np.zeros((M, O), bool)
    bad[M // 2, :] = True
    bad[:, 200] = True
    assert np.isnan(y[bad]).all() and np.array_equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("M", [1, 2, 20, 300])
def test_zero_scale_rows_and_zero_tokens(lib, torch, M):
    """s = 0 leaves the rank term alone; a token of zeros gives zeros."""
    p = Problem(lib, torch, M, 136, 272, 8)
    p.s[:] = np.where(np.arange(136) % 3 == 0, 0.0, p.s)
    p.sd.copy_(dev(p.s))
    p.X[M // 2] = 0.0
    p.Xd.copy_(dev(p.X, "bf16"))
    p.xc, p.xs = encode_rows(lib, torch, p.Xd)
    y = host(p.call())
    lib.theta_device_status()
    p.check()
    assert not y[M // 2].any()


def test_31b_gate_on_sampled_rows(lib, torch):
    O, I = syn.GEMMA4_31B.shapes["gate"]
    r = 64
    rows = np.sort(np.random.default_rng(3).choice(O, 24, replace=False))
    wc, ws = encode(lib, torch, syn.device_normal((O, I), 0.02, 0, "W0", "fp8-31b"))
    for M in (1, 2, 16, 700):
        p = Problem(lib, torch, M, 8, I, r)  # the tokens and V
        p.dims = (M, O, I, r)
        p.wc, p.ws = wc, ws
        p.sd = 1.0 + syn.device_normal((O,), 0.05, 0, "s", "fp8-31b", dtype="f32")
        p.Ud = syn.device_normal((O, r), 0.05, 0, "U", "fp8-31b")
        p.s, p.U = p.sd.cpu().numpy(), host(p.Ud)
        p.guard = torch.full((M * O + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        p.Y = p.guard[256:256 + M * O].view(M, O)
        nb = lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, M, O, I, r, lib.THETA_BF16)
        p.work = torch.empty(nb, dtype=torch.uint8, device="cuda")
        p.call()
        lib.theta_device_status()
        # the sampled rows of W0 only, with their blocks' scales
        w = oracle.fp8_values(wc[torch.from_numpy(rows).cuda()].cpu().numpy())
        w = w * np.repeat(np.exp2(ws.cpu().numpy()[rows // 128].astype(float) - 127), 128, axis=1)[:, :I]
        p.values = lambda rows, x=oracle.fp8_dequantize_rows(p.xc.cpu().numpy(), p.xs.cpu().numpy()): (x, w)
        p.check(rows=rows, what=f"M={M}")


# ------------------------------------------------------------------ how it is called
@pytest.mark.parametrize("M", [1, 2, 24, 300])
def test_captured_and_replayed_and_on_another_stream(lib, torch, M):
    p = Problem(lib, torch, M, 520, 656, 16)
    want = p.call().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.Y.fill_(0)
        p.call()
    side.synchronize()
    assert torch.equal(p.Y, want)
    p.Y.fill_(0)
    p.call(stream=side)
    side.synchronize()
    assert torch.equal(p.Y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.theta_fp8_quantize_rows(p.Xd, p.xc, p.xs)
        p.call()
    for k in range(2):
        p.X = oracle.round_to(np.roll(p.X, 1 + k, axis=1), "bf16").astype(np.float32)
        p.Xd.copy_(dev(p.X, "bf16"))
        g.replay()
        lib.theta_device_status()
        p.check(what=f"replay {k}")


@pytest.mark.parametrize("M", [1, 16, 300])
def test_work_after_a_timeout_is_flagged_then_recovers(lib, torch, M):
    """A forward enqueued while the timeout flag is set gives up within its
    bounded waits; the next one, after the flag has been read, is right."""
    p = Problem(lib, torch, M, 520, 656, 16)
    lib.theta_device_status()
    lib.theta_selftest_wait_timeout(20)
    p.call()
    with pytest.raises(lib.ThetaError) as err:
        lib.theta_device_status()
    assert err.value.status == -5
    p.call()
    lib.theta_device_status()
    p.check()


@pytest.mark.parametrize("M,O,r", [(1000, 8200, 0), (1000, 8200, 8), (300, 21504, 0)])
@pytest.mark.parametrize("I", [16, 272, 512, 640, 656, 896, 1168])
def test_scale_groups_over_several_tiles_of_a_cluster(lib, torch, M, O, r, I):
    """More CTA-pair tiles than pairs, with and without a rank term between
    them, the last scale group of a tile of 1 to 4 blocks; every block of W0
    and every token's block has a scale far from its neighbours', so that one
    used for another shows."""
    p = Problem(lib, torch, M, O, I, r)
    g = torch.Generator(device="cuda").manual_seed(I)
    for scales in (p.xs, p.ws):
        scales.copy_(torch.randint(117, 138, scales.shape, device="cuda", generator=g))
    p.call()
    lib.theta_device_status()
    p.check(what=f"{M}x{O}x{I} r{r}")


@pytest.mark.parametrize("sized_for", [2, 3, 16, 64, 300])
def test_one_workspace_for_a_batch_that_shrinks(lib, torch, sized_for):
    """A buffer sized for a batch serves smaller ones, down to one token, and
    nothing behind it is written."""
    O, I, r = 264, 656, 64
    nb = lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, sized_for, O, I, r, lib.THETA_BF16)
    buf = torch.full((nb + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for M in sorted({m for m in (sized_for, 64, 16, 3, 2, 1) if m <= sized_for}, reverse=True):
        p = Problem(lib, torch, M, O, I, r)
        p.work = buf[:nb]
        p.call()
        lib.theta_device_status()
        p.check(what=f"{M} of {sized_for} tokens")
        assert (buf[nb:] == 0xA5).all()


def test_outputs_past_32_bit_offsets(lib, torch):
    """Y, and the row encoder's input and codes, of more than 2^31 elements."""
    M, O, I = 131072, 21504, 16
    p = Problem(lib, torch, 8, O, I, 8)
    X = p.Xd.repeat(M // 8, 1)
    xc, xs = encode_rows(lib, torch, X)
    Y = torch.empty(M, O, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, M, O, I, 8, lib.THETA_BF16),
                       dtype=torch.uint8, device="cuda")
    lib.theta_linear_forward_fp8(X, xc, xs, p.wc, p.ws, p.sd, p.Ud, p.Vd, Y, work)
    lib.theta_device_status()
    for at in (0, M // 2, M - 8):
        p.check(Y=Y[at:at + 8], what=f"tokens from {at}")
    del X, xc, xs, Y
    M, I = 40000, 65536
    X = torch.randn(8, I, device="cuda").bfloat16().repeat(M // 8, 1)
    c, s = encode_rows(lib, torch, X)
    lib.theta_device_status()
    cr, sr = oracle.fp8_quantize_rows(host(X[:8]))
    for at in (0, M - 8):
        assert np.array_equal(c[at:at + 8].cpu().numpy(), cr) and np.array_equal(s[:, at:at + 8].cpu().numpy(), sr)


def test_two_calls_at_once_on_two_streams(lib, torch):
    ps = [Problem(lib, torch, M, 1032, 1168, 16, seed=M) for M in (1, 40, 300, 1, 40, 300)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, st in zip(ps, streams):
            p.call(stream=st)
    torch.cuda.synchronize()
    lib.theta_device_status()
    for p in ps:
        p.check()


def test_first_calls_of_fresh_threads(lib, torch):
    """Several host threads, each making its first CUDA call through the
    library, on streams of their own: FP8 and bf16 forwards."""
    import threading
    ps = [Problem(lib, torch, M, 520, 656, 16, seed=M) for M in (1, 2, 40, 300, 40, 300)]
    streams = [torch.cuda.Stream() for _ in ps]
    X, W = torch.randn(40, 656, device="cuda").bfloat16(), torch.randn(520, 656, device="cuda").bfloat16()
    s, Y = torch.ones(520, device="cuda"), torch.zeros(40, 520, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    failed = []

    def guarded(call):
        try:
            for _ in range(10):
                call()
        except Exception as e:  # noqa: BLE001 - reported below
            failed.append(e)
    calls = [lambda p=p, st=st: p.call(stream=st.cuda_stream) for p, st in zip(ps, streams)]
    side = torch.cuda.Stream()
    calls.append(lambda: lib.theta_linear_forward(X, W, s, None, None, Y, None, stream=side.cuda_stream))
    threads = [threading.Thread(target=guarded, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    lib.theta_device_status()
    assert not failed, failed
    for p in ps:
        p.check()
    ref = host(X) @ host(W).T
    assert np.abs(host(Y) - ref).max() <= 2e-2 * np.sqrt(np.mean(ref ** 2))


@pytest.mark.parametrize("what", ["blocks", "rows", "forward 1", "forward 4", "forward 300", "heads"])
def test_first_call_of_a_process_captured(what):
    """A process whose first call of the library is made inside a graph capture."""
    import os
    import subprocess
    import sys
    code = """
import sys, torch
import linear_theta_forward_b200 as th
op, M, bf = sys.argv[1], int(sys.argv[2]), torch.bfloat16
r = lambda *s: torch.randn(*s, device="cuda").to(bf)
z = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")
W, X, U, V, s, Q = r(256, 400), r(M, 400), r(256, 16), r(400, 16), torch.ones(256, device="cuda"), r(M, 256)
wc, ws, xc, xs = z(256, 400) % 64, z(2, 4), z(M, 400) % 64, z(4, M)
Y, Qo = torch.zeros(M, 256, dtype=bf, device="cuda"), torch.zeros_like(Q)
work, pos, f = z(1 << 18), torch.arange(M, device="cuda"), torch.ones(32, device="cuda")
call, out = {"blocks": (lambda: th.theta_fp8_quantize(W, wc, ws), wc),
             "rows": (lambda: th.theta_fp8_quantize_rows(X, xc, xs), xc),
             "forward": (lambda: th.theta_linear_forward_fp8(X, xc, xs, wc, ws, s, U, V, Y, work), Y),
             "heads": (lambda: th.theta_qk_norm_rope(Q, None, None, None, pos, f, Qo, None, 64), Qo)}[op]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
th.theta_device_status()
a = out.clone()
out.zero_()
call()
th.theta_device_status()
assert torch.equal(a, out) and a.float().abs().sum() > 0
"""
    op, _, m = what.partition(" ")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code, op, m or "4"], cwd=root, timeout=120, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]


def test_attention_inputs_together(lib, torch):
    """One token batch quantized once, the q and k projections over it in FP8,
    the heads normed and rotated in place -- against the oracle's chain, each
    step from the GPU's own output of the step before."""
    M, I, D, r = 37, 1152, 256, 32
    hq, hk = 4, 1
    q, k = Problem(lib, torch, M, hq * D, I, r, seed=5), Problem(lib, torch, M, hk * D, I, r, seed=6)
    k.X, k.Xd, k.xc, k.xs = q.X, q.Xd, q.xc, q.xs
    wq, wk = syn.host_normal((D,), 0.1, 1, "wq", dtype="bf16"), syn.host_normal((D,), 0.1, 1, "wk", dtype="bf16")
    pos = torch.arange(1000, 1000 + M, device="cuda")
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float32) / (D // 2))).cuda()
    q.call(), k.call()
    q.check(), k.check()
    yq, yk = host(q.Y), host(k.Y)
    lib.theta_qk_norm_rope(q.Y, k.Y, dev(wq, "bf16"), dev(wk, "bf16"), pos, freq, q.Y, k.Y, D, weight_offset=1.0)
    lib.theta_device_status()
    for y, got, w in ((yq, q.Y, wq), (yk, k.Y, wk)):
        ref = oracle.qk_norm_rope(y, D, w, 1.0, 1e-6, pos.cpu().numpy(), freq.cpu().numpy(), False)
        mag = np.sqrt(2.0) * np.abs(oracle.qk_norm_rope(y, D, w, 1.0, 1e-6, pos.cpu().numpy(), None, False)).max()
        assert np.all(np.abs(host(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (24 + D / 16) * 2.0 ** -24 * mag)
    assert (q.guard[:256] == 7).all() and (q.guard[256 + M * hq * D:] == 7).all()


def test_in_place_refusal_leaves_memory_alone(lib, torch):
    p = Problem(lib, torch, 4, 16, 64, 8)
    with pytest.raises(lib.ThetaError):
        lib.theta_linear_forward_fp8(p.Xd, p.xc, p.xs, p.wc, p.ws, p.sd, p.Ud, p.Vd, p.Y, None)  # no workspace
    with pytest.raises(ValueError):
        lib.theta_linear_forward_fp8(p.Xd, p.xc, p.xs.view(4, 1), p.wc, p.ws, p.sd, p.Ud, p.Vd, p.Y, p.work)
    with pytest.raises(ValueError):
        lib.theta_linear_forward_fp8(p.Xd.float(), p.xc, p.xs, p.wc, p.ws, p.sd, p.Ud, p.Vd, p.Y, p.work)
    torch.cuda.synchronize()
    assert (p.guard == 7).all()
