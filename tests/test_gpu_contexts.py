"""Which CUDA context a call works in: the one that is current in its thread,
and the device's primary context only where there is none.

Each case runs in a process of its own that uses the driver API directly, so
that no other library has made a context current."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

COMMON = """
import ctypes, sys
import numpy as np
import oracle
import linear_theta_forward_b200 as th
raw, cu = th.lib, ctypes.CDLL("libcuda.so.1")
u64, vp = ctypes.c_uint64, ctypes.c_void_p

def ok(status):
    assert status == 0, f"driver status {status}"

def current():
    c = vp()
    ok(cu.cuCtxGetCurrent(ctypes.byref(c)))
    return c.value

def create():
    c = vp()
    ok(cu.cuCtxCreate_v2(ctypes.byref(c), 0, 0))
    return c

def primary():
    c = vp()
    ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(c), 0))
    return c

def upload(a):
    a = np.ascontiguousarray(a)
    p = u64()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(a.nbytes)))
    ok(cu.cuMemcpyHtoD_v2(p, vp(a.ctypes.data), ctypes.c_size_t(a.nbytes)))
    return vp(p.value)

def download(p, shape, dtype):
    a = np.empty(shape, dtype)
    ok(cu.cuMemcpyDtoH_v2(vp(a.ctypes.data), u64(p.value), ctypes.c_size_t(a.nbytes)))
    return a

def stream():
    s = vp()
    ok(cu.cuStreamCreate(ctypes.byref(s), 1))  # does not wait for the default stream
    return s

def bits(a):  # bf16 of values that bf16 holds
    return (np.asarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16)

class Case:
    \"\"\"An encoder and the bf16 forwards (TMA descriptors; built-in scratch) in the context that is current.\"\"\"
    O, I, r, M = 264, 400, 16, 40

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        bf = lambda *s: oracle.round_to(rng.standard_normal(s), "bf16").astype(np.float32)
        self.X, self.W, self.U, self.V = bf(self.M, self.I), bf(self.O, self.I), bf(self.O, self.r), bf(self.I, self.r)
        self.s = np.linspace(0.5, 1.5, self.O).astype(np.float32)
        self.stream = stream()
        self.dev = [upload(bits(a)) for a in (self.X, self.W, self.U, self.V)]
        self.ds = upload(self.s)
        self.codes, self.scales = upload(np.zeros((self.O, self.I), np.uint8)), upload(np.zeros((3, 4), np.uint8))
        self.Y = [upload(np.zeros((self.M, self.O), np.uint16)) for _ in range(2)]
        self.work = upload(np.zeros(1 << 16, np.uint8))
        ok(cu.cuCtxSynchronize())

    def run(self):
        X, W, U, V = self.dev
        o, i, r, m, st = self.O, self.I, self.r, self.M, self.stream
        for status in (raw.theta_fp8_quantize(W, o, i, 1, self.codes, self.scales, st),
                       raw.theta_linear_forward(X, m, i, W, o, self.ds, U, V, r, 1, self.Y[0], self.work, 1 << 16, st),
                       raw.theta_linear_forward_noalloc(X, m, i, W, o, self.ds, U, V, r, 1, self.Y[1], st),
                       raw.theta_device_status(st)):
            assert status == 0, (status, th.theta_last_error())
        cr, sr = oracle.fp8_quantize(self.W)
        assert np.array_equal(download(self.codes, (o, i), np.uint8), cr)
        assert np.array_equal(download(self.scales, (3, 4), np.uint8), sr)
        ref = oracle.linear_forward(self.X, self.W, self.s, self.U, self.V)
        for y in self.Y:
            got = (download(y, (m, o), np.uint16).astype(np.uint32) << 16).view(np.float32)
            assert np.abs(got - ref).max() <= 2e-2 * np.sqrt(np.mean(ref ** 2))

ok(cu.cuInit(0))
"""

CASES = {
    # every entry point finds its context before it looks at what only the
    # kernels can refuse: this one is refused there, and nothing is launched
    "a refused call leaves the caller's context current": """
mine = create()
assert current() == mine.value
P = vp(4096)
assert raw.theta_linear_forward_nvfp4(P, 1, 1 << 20, P, P, P, 8, P, None, None, 0, P, None, 0, None) == -2
assert current() == mine.value
""",
    "calls in a context of the caller's own": """
mine = create()
case = Case(1)
for _ in range(2):
    case.run()
    assert current() == mine.value
""",
    "a thread whose context is taken off between calls": """
p = primary()
ok(cu.cuCtxSetCurrent(p))
case = Case(2)
case.run()
ok(cu.cuCtxSetCurrent(None))
X, W, U, V = case.dev
for _ in range(2):  # descriptors to encode, on a thread that has bound the context before
    assert raw.theta_linear_forward(X, case.M, case.I, W, case.O, case.ds, U, V, case.r, 1, case.Y[0], case.work,
                                    1 << 16, case.stream) == 0, th.theta_last_error()
    assert current() == p.value
    ok(cu.cuCtxSetCurrent(None))
ok(cu.cuCtxSetCurrent(p))
case.run()
""",
    "calls in turn in several contexts of one device": """
contexts = [primary(), create(), create()]
cases = []
for n, c in enumerate(contexts):
    ok(cu.cuCtxSetCurrent(c))
    cases.append(Case(3 + n))
for _ in range(2):
    for c, case in zip(contexts, cases):
        ok(cu.cuCtxSetCurrent(c))
        case.run()
        assert current() == c.value
ok(cu.cuCtxDestroy_v2(contexts.pop()))
last = create()  # where the destroyed one may have been
Case(9).run()
ok(cu.cuCtxSetCurrent(contexts[0]))
cases[0].run()
""",
    "a timeout is reported in its own context": """
contexts = [primary(), create()]
cases = []
for n, c in enumerate(contexts):
    ok(cu.cuCtxSetCurrent(c))
    cases.append(Case(20 + n))
    cases[n].run()
assert raw.theta_selftest_wait_timeout(20, cases[1].stream) == 0
assert raw.theta_device_status(cases[1].stream) == -5
for c, case in zip(contexts, cases):
    ok(cu.cuCtxSetCurrent(c))
    case.run()
""",
}


def run_case(code, limit=120):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", COMMON + code], cwd=root, timeout=limit, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.parametrize("what", list(CASES))
def test_context_of_a_call(what):
    run_case(CASES[what])


LAST = """
P = vp(4096)
call = lambda: raw.theta_linear_forward_nvfp4(P, 1, 1 << 20, P, P, P, 8, P, None, None, 0, P, None, 0, None)
first = create()
case = Case(30)
case.run()
for n in range(64):
    c = create()
    assert call() == -2
    assert ("contexts" in th.theta_last_error()) == (n == 63), (n, th.theta_last_error())
    assert current() == c.value
    ok(cu.cuCtxDestroy_v2(c))
    ok(cu.cuCtxSetCurrent(first))
case.run()
"""


@pytest.mark.slow
def test_context_after_the_last_is_refused():
    """64 contexts are served and the next one refused, with the first still
    served (each context loads the library's kernels: about 45 s)."""
    run_case(LAST, limit=600)
