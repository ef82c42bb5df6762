"""A handle-free operator's first call on a device sets all of its variants up: calls of other sizes
and types may then be captured without a call of their own before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# in a fresh process: one small call of each operator, then a capture of calls that take every other
# variant; the kernels are whole-number sums, exact
CODE = r"""
import torch, mixture_experts_ffn_rmsnorm_b200 as moe
gen = torch.Generator(device="cuda").manual_seed(1)
BF, HF = torch.bfloat16, torch.float16
def ints(*s, dt=BF):
    return torch.randint(-1, 2, s, device="cuda", generator=gen).to(dt)
def off(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")
x, w, y, o = ints(4, 64), ints(2, 48, 64), ints(4, 48), off(0, 1, 4)
moe.grouped_gemm(x, w, o, torch.zeros_like(y))
moe.grouped_gemm_dgrad(y, w, o, torch.zeros_like(x))
moe.grouped_gemm_wgrad(y, x, o, torch.zeros_like(w))
def fp4(E, N, K):
    return (torch.full((E, N, K // 2), 0x22, dtype=torch.uint8, device="cuda"),
            torch.full((E, N, K // 16), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(E, device="cuda"))
ids = off(1).view(1, 1)
moe.nvfp4_gemv(ints(1, 32), ids, *fp4(2, 16, 32), torch.zeros(1, 1, 16, dtype=BF, device="cuda"))
torch.cuda.synchronize()

R = 2600
X, D, W = ints(R, 2048), ints(R, 2304), ints(1, 2304, 2048)
x2, d2, w2 = ints(600, 2048), ints(600, 2304), ints(6, 2304, 2048)
o1, o6 = off(0, R), off(0, 100, 200, 300, 400, 500, 600)
Y, DX, DW, DF = (torch.zeros_like(t) for t in (D, X, W, W.float()))
y2, dx2 = torch.zeros_like(d2), torch.zeros_like(x2)
sf = torch.zeros(2, 48, 64, device="cuda")
cases = [(dt, K, ints(1, K, dt=dt), fp4(2, 16, K), torch.zeros(1, 1, 16, dtype=dt, device="cuda"))
         for dt in (BF, HF) for K in (256, 128, 64, 32)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, capture_error_mode="global"):
    moe.grouped_gemm(X, W, o1, Y)
    moe.grouped_gemm(x2, w2, o6, y2)
    moe.grouped_gemm_dgrad(D, W, o1, DX)
    moe.grouped_gemm_dgrad(d2, w2, o6, dx2)
    moe.grouped_gemm_wgrad(D, X, o1, DW)
    moe.grouped_gemm_wgrad(D, X, o1, DF)
    moe.grouped_gemm_wgrad(y, x, o, sf)
    for dt, K, t, f, out in cases:
        moe.nvfp4_gemv(t, ids, *f, out)
graph.replay()
torch.cuda.synchronize()
f = lambda t: t.float()
assert torch.equal(Y, (f(X) @ f(W[0]).T).to(BF)) and torch.equal(DX, (f(D) @ f(W[0])).to(BF))
assert torch.equal(DF[0], f(D).T @ f(X)) and torch.equal(DW[0], DF[0].to(BF))
for e in range(6):
    s = slice(100 * e, 100 * e + 100)
    assert torch.equal(y2[s], (f(x2[s]) @ f(w2[e]).T).to(BF)) and torch.equal(dx2[s], (f(d2[s]) @ f(w2[e])).to(BF))
assert torch.equal(sf[1], f(y[1:]).T @ f(x[1:]))
for dt, K, t, f4, out in cases:
    assert (out == t.float().sum()).all()
graph.reset()
print("ok")
"""


@pytest.mark.parametrize("loading", ("LAZY", "EAGER"))
def test_first_calls_set_every_variant_up(loading):
    env = dict(os.environ, CUDA_MODULE_LOADING=loading)
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
