"""Waits inside the kernels for a few tokens that run out: an error that the host reads, and calls after it as if it had not been.

With a limit of 0 a role gives up at the first thing that is not there yet, while the copies of all stages are under way.
"""
import pytest
import torch

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L

pytestmark = pytest.mark.gpu
NEVER = 2_000_000_000


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


def make(bits, *shape):
    w = (torch.randn(shape, device="cuda") * 0.05).bfloat16()
    return L.mx4_quantize(w) if bits == 4 else L.mx_quantize_experts(w if w.dim() == 3 else w[None], colwise=False)


class Linear:
    def __init__(self, M, N, K, bits):
        torch.manual_seed(M + N + K + bits)
        self.x = torch.randn(M, K, device="cuda").bfloat16()
        self.q, self.e8, self.bits = L._held(make(bits, 1, N, K))
        self.ws = torch.empty(FB.mx_few_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")

    def args(self):
        y = torch.empty(self.x.shape[0], self.q.shape[1], dtype=torch.bfloat16, device="cuda")
        return self.x, self.q[0], self.e8, self.bits, y, self.ws if len(self.ws) else None

    def run(self):
        args = self.args()
        FB.mx_few_linear(*args)
        return args[4]

    def selftest(self, wait_ns):
        args = self.args()
        FB.fp8bw_selftest_few_linear(*args, wait_ns=wait_ns)
        return args[4]


class Layer:
    def __init__(self, M, E, k, C, F, bits):
        torch.manual_seed(M + E + k + C + F + bits)
        self.x, self.k = torch.randn(M, C, device="cuda").bfloat16(), k
        self.router = torch.randn(E, C, device="cuda") / C ** 0.5
        self.q13, self.e13, self.bits = L._held(make(bits, E, 2 * F, C))
        self.q2, self.e2, _ = L._held(make(bits, E, C, F))
        self.ws = torch.empty(FB.mx_few_moe_workspace_bytes(M, E, k, C, F), dtype=torch.uint8, device="cuda")

    def args(self):
        return (self.x, self.router, None, self.q13, self.e13, self.q2, self.e2, self.bits, self.k, torch.empty_like(self.x), self.ws)

    def run(self):
        args = self.args()
        FB.mx_few_moe(*args)
        return args[9]

    def selftest(self, wait_ns):
        args = self.args()
        FB.fp8bw_selftest_few_moe(*args, wait_ns=wait_ns)
        return args[9]


def status():
    try:
        B.fp8bw_sync_status()
    except B.Fp8bwError as e:
        return e.code
    return 0


LINEARS = [(1, 2048, 2048, 4), (2, 8192, 5120, 8), (5, 3001, 7136, 4), (8, 1024, 8192, 8), (32, 8192, 5120, 4), (32, 640, 1056, 4)]
LAYERS = [(1, 8, 2, 2048, 1024, 4), (5, 4, 2, 1056, 672, 4), (17, 64, 4, 1024, 512, 4), (32, 8, 2, 1024, 2048, 8), (32, 1, 1, 512, 512, 8)]
CASES = [(Linear, c) for c in LINEARS] + [(Layer, c) for c in LAYERS]


@pytest.mark.parametrize("kind,case", CASES, ids=lambda v: v.__name__ if isinstance(v, type) else "-".join(map(str, v)))
def test_a_wait_that_runs_out(kind, case):
    c = kind(*case)
    want = c.run()
    assert status() == 0
    assert torch.equal(c.selftest(NEVER), want) and status() == 0
    c.selftest(0)
    assert status() == B.ERR_TIMEOUT
    assert status() == 0  # read and cleared
    assert torch.equal(c.run(), want) and status() == 0
    for wait_ns in (200, 1000, 4000):  # somewhere on the way, or not at all
        got = c.selftest(wait_ns)
        assert status() in (0, B.ERR_TIMEOUT) and got.shape == want.shape
    for _ in range(10):  # right behind blocks that gave up, on the same multiprocessors
        for _ in range(3):
            c.selftest(0)
        got = c.run()
        assert status() == B.ERR_TIMEOUT and torch.equal(got, want)


def test_others_right_behind():
    """Blocks of another kernel get the shared memory of those that gave up, while those run."""
    cases = [kind(*case) for kind, case in CASES]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    for i, first in enumerate(cases):
        for j, second in enumerate(cases):
            first.selftest(0)
            got = second.run()
            torch.cuda.synchronize()
            assert torch.equal(got, want[j]), (i, j)
    assert status() == B.ERR_TIMEOUT


def test_refusals():
    c = Linear(2, 64, 64, 4)
    with pytest.raises(B.Fp8bwError):
        c.selftest(NEVER + 1)
    d = Layer(2, 4, 2, 64, 64, 4)
    with pytest.raises(B.Fp8bwError):
        d.selftest(NEVER + 1)
