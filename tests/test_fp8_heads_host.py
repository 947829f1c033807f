"""Block-scaled FP8 and the per-head norm with rotation without a GPU: the
oracle against independent readings of the formats and formulas, and the C
ABI's and the binding's refusals (nothing reaches the CUDA runtime)."""
import ctypes

import numpy as np
import pytest

import oracle

P = ctypes.c_void_p(4096)  # a 16-byte aligned fake device address: validation fails before any launch
ODD = ctypes.c_void_p(4100)


# ------------------------------------------------------------------ the oracle
def test_e4m3_rounding_matches_torch():
    import torch
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-4, 2, 4000), [448.0, -448.0, 0.0, 2.0 ** -9,
                        2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 0.0625 * 1.0625]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    code = oracle._grid_round(np.abs(x), oracle.e4m3_values()) | np.where(np.signbit(x), 128, 0)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(code, t)
    assert np.array_equal(oracle.fp8_values(t), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("a,e", [(448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.7500001, -7),
                                 (0.0, 0), (1e-45, -127), (3.4e38, 120)])
def test_block_exponent(a, e):
    assert oracle.theta_oracle._fp8_exponent(float(np.float32(a))) == e


def test_encodings_stay_within_half_a_step_and_hide_nothing():
    rng = np.random.default_rng(2)
    W = rng.standard_normal((150, 304)) * 10.0 ** rng.uniform(-3, 3, (150, 1))
    W[3, 7], W[140, 300] = np.inf, np.nan
    W[128:, 128:256] = 0.0
    c, s = oracle.fp8_quantize(W)
    assert s.shape == (2, 3) and s[1, 1] == 127 and not c[128:, 128:256].any()
    assert c[3, 7] == 127 and c[140, 300] == 127
    D = oracle.fp8_dequantize(c, s)
    ok = np.isfinite(W)
    block = np.exp2(np.repeat(np.repeat(s.astype(float) - 127, 128, 0)[:150], 128, 1)[:, :304])
    assert np.all(np.abs(D - W)[ok] <= np.maximum(2.0 ** -4 * np.abs(W), 2.0 ** -10 * block)[ok])
    assert np.isnan(D[~ok]).all()
    x, xs = oracle.fp8_quantize_rows(W[:5])
    assert xs.shape == (3, 5)
    for m in range(5):  # a row alone is a block of one row
        c1, s1 = oracle.fp8_quantize(W[m:m + 1])
        assert np.array_equal(c1[0], x[m]) and np.array_equal(s1[0], xs[:, m])


def test_rotation_keeps_length_and_composes():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2 * 16))
    f = 10000.0 ** (-np.arange(6) / 6.0)
    for inter in (False, True):
        y = oracle.qk_norm_rope(x, 16, None, 0.0, 0.0, np.array([0, 1, 2, 50]), f, inter)
        h = y.reshape(4, 2, 16)
        assert np.allclose((h ** 2).sum(2), 16.0)          # unit RMS, lengths kept by the rotation
        assert np.allclose(y[0], oracle.qk_norm_rope(x, 16, None, 0.0, 0.0, [0] * 4, None, inter)[0])
        # products of queries and keys depend on the distance of the positions only
        q, k = x[:1], x[1:2]
        dot = [oracle.qk_norm_rope(q, 16, None, 0, 0, [a], f, inter)[0, :16] @
               oracle.qk_norm_rope(k, 16, None, 0, 0, [b], f, inter)[0, :16] for a, b in ((3, 1), (103, 101))]
        assert np.isclose(dot[0], dot[1])


# ------------------------------------------------------------------ refusals
def test_quantize_refusals(lib):
    raw = lib.lib
    for f in (raw.theta_fp8_quantize, raw.theta_fp8_quantize_rows):
        assert f(P, 0, 64, 1, P, P, None) == -1
        assert f(P, 8, 0, 1, P, P, None) == -1
        assert f(P, 8, 64, 7, P, P, None) == -1              # dtype
        assert f(None, 8, 64, 1, P, P, None) == -1
        assert f(P, 8, 64, 1, None, P, None) == -1
        assert f(P, 8, 64, 1, P, None, None) == -1
        assert f(P, 8, 72, 1, P, P, None) == -3              # I % 16
        assert f(ODD, 8, 64, 1, P, P, None) == -3
        assert f(P, 8, 64, 0, ODD, P, None) == -3
        assert f(P, 1 << 40, 64, 1, P, P, None) == -2
        assert f(P, 1 << 20, 1 << 29, 1, P, P, None) == -2   # more blocks than a grid holds


def test_forward_refusals(lib):
    raw = lib.lib

    def call(X=P, xq=P, xs=P, M=4, I=64, wq=P, ws=P, O=8, s=P, U=P, V=P, r=8, Y=P, work=P, nbytes=1 << 20):
        return raw.theta_linear_forward_fp8(X, xq, xs, M, I, wq, ws, O, s, U, V, r, Y, work, nbytes, None)
    for bad in (dict(M=0), dict(I=0), dict(O=0), dict(r=-1), dict(r=264), dict(xq=None), dict(xs=None),
                dict(wq=None), dict(ws=None), dict(s=None), dict(Y=None), dict(X=None), dict(U=None), dict(V=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(I=72), dict(O=12), dict(r=12), dict(X=ODD), dict(xq=ODD), dict(wq=ODD), dict(s=ODD),
                dict(U=ODD), dict(V=ODD), dict(Y=ODD)):
        assert call(**bad) == -3, bad
    for bad in (dict(M=65535 * 64 + 1), dict(O=65535 * 64 + 8), dict(I=1 << 30)):
        assert call(nbytes=1 << 60, **bad) == -2, bad
    need = lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, 4, 8, 64, 8, lib.THETA_BF16)
    assert need > 0 and call(nbytes=need - 1) == -6 and call(work=None) == -6 and call(work=ODD) == -6
    assert lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, 4, 8, 64, 0, lib.THETA_BF16) == 0
    for M, r in ((0, 8), (4, -1), (4, 300)):
        with pytest.raises(lib.ThetaError):
            lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, M, 8, 64, r, lib.THETA_BF16)


def test_forward_workspace_does_not_fall_as_tokens_or_rank_grow(lib):
    """One buffer, sized for the largest batch, serves every smaller one."""
    counts = [*range(1, 70), 127, 128, 129, 240, 241, 2048, 100000]
    table = [[lib.theta_workspace_size(lib.THETA_OP_LINEAR_FORWARD_FP8, M, 8, 64, r, lib.THETA_BF16)
              for r in (0, 8, 24, 32, 64, 200, 256)] for M in counts]
    assert all(a <= b for small, large in zip(table, table[1:]) for a, b in zip(small, large))
    assert all(a <= b for sizes in table for a, b in zip(sizes, sizes[1:]))


def test_heads_refusals(lib):
    raw = lib.lib

    def call(Q=P, ldq=512, hq=2, K=P, ldk=256, hk=1, M=4, D=256, dt=1, wq=P, wk=P, off=0.0, eps=1e-6, pos=P, f=P,
             rot=256, inter=0, Qo=P, ldqo=512, Ko=P, ldko=256):
        return raw.theta_qk_norm_rope(Q, ldq, hq, K, ldk, hk, M, D, dt, wq, wk, off, eps, pos, f, rot, inter, Qo, ldqo,
                                      Ko, ldko, None)
    for bad in (dict(M=0), dict(M=(1 << 30) + 1), dict(hq=0), dict(hq=65536), dict(hk=-1), dict(hk=65536), dict(D=0),
                dict(D=12), dict(rot=-2), dict(rot=258), dict(rot=7), dict(eps=-1.0), dict(eps=float("nan")),
                dict(dt=3), dict(Q=None), dict(Qo=None), dict(K=None), dict(Ko=None), dict(pos=None), dict(f=None),
                dict(ldq=504), dict(ldqo=504), dict(ldk=248), dict(ldko=0), dict(ldqo=520), dict(ldko=264)):
        assert call(**bad) == -1, bad
    assert call(D=1032, rot=0, ldq=4096, ldqo=4096, ldk=4096, ldko=4096) == -2
    for bad in (dict(wq=ODD), dict(wk=ODD), dict(Q=ODD), dict(Qo=ODD), dict(K=ODD), dict(Ko=ODD), dict(ldq=516, ldqo=516), dict(pos=ODD),
                dict(f=ctypes.c_void_p(4098))):
        assert call(**bad) == -3, bad


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    import torch
    W = torch.zeros(8, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        lib.theta_fp8_quantize(W, c, s)
    with pytest.raises(ValueError, match="CUDA"):
        lib.theta_fp8_quantize_rows(W, c, s)
    with pytest.raises(ValueError, match="CUDA"):
        lib.theta_qk_norm_rope(W, None, None, None, None, None, W, None, 64)
    with pytest.raises(ValueError, match="together"):
        lib.theta_linear_forward_fp8(None, c, s, c, s, None, W, None, W)
    with pytest.raises(ValueError, match="X_codes|codes"):
        lib.theta_linear_forward_fp8(None, W, s, c, s, None, None, None, W)
