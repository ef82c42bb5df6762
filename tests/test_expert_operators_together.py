"""The handle-free expert operators in the order they are used: a training step of
routed experts on the library's own sort, and a decode step on NVFP4 experts with
the layer's own routing, replayed from a CUDA graph.

The references are the same formulas in 64 bits.  Each step's error bound is carried
through the next one: a product of a matrix with an operand that is off by d is off by
at most |matrix| d, plus q * 2^-23 (|matrix| |operand|) for its own float32 sums, plus
half a step of the output's type (2^-8 for BF16); relu^2 of h off by d by 2 |h| d + d^2;
its derivative 2 relu(h) by 2 d.
"""
import numpy as np
import pytest

from workloads import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA device", allow_module_level=True)

import mixture_experts_ffn_rmsnorm_b200 as moe  # noqa: E402

HALF = 2.0 ** -8   # half a BF16 step, relative
SUM = 2.0 ** -23   # of a float32 addition, truncation allowed


def rounded(ref, err):
    return err + HALF * (ref.abs() + err) + 1e-38


def product(A, dA, B, dB):
    """(A @ B, bound of its error) for operands off by dA and dB."""
    a, b = A.abs() + dA, B.abs() + dB
    return A @ B, dA @ B.abs() + A.abs() @ dB + dA @ dB + A.shape[-1] * SUM * (a @ b)


def check(got, ref, err, what):
    bad = (got.double() - ref).abs() > err
    assert not bad.any(), (what, int(bad.sum()))


def test_training_step_of_routed_experts():
    T, k, E, H, I = 300, 3, 16, 192, 136
    gen = torch.Generator(device="cuda").manual_seed(21)
    bf = torch.bfloat16
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, g = r(T, H).to(bf), r(T, H).to(bf)
    up, down = (r(E, I, H) * H ** -0.5).to(bf), (r(E, H, I) * I ** -0.5).to(bf)
    idx = torch.rand(T, E, device="cuda", generator=gen)
    idx[:, 3] = 0  # an expert without rows
    idx = idx.topk(k, dim=1).indices.to(torch.int32)
    wts = torch.rand(T, k, device="cuda", generator=gen)
    R = T * k
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    perm, inv, off = z(R, dt=torch.int32), z(R, dt=torch.int32), z(E + 1, dt=torch.int32)
    status = z(1, dt=torch.int32)

    # forward: sort, gather, up, relu^2, down, weighted sum
    moe.sort_static(idx, k, E, perm, inv, off)
    token = perm.long() // k
    xs = x[token]
    h, a, y = z(R, I), z(R, I), z(R, H)
    moe.grouped_gemm(xs, up, off, h, status=status)
    moe.grouped_gemm(xs, up, off, a, relu2=True, status=status)
    moe.grouped_gemm(a, down, off, y, status=status)
    # backward of sum(g * out) down to the weights and the gathered rows
    dy = (g[token].float() * wts.flatten()[perm.long()].unsqueeze(1)).to(bf)
    da, dxs = z(R, I), z(R, H)
    d_up, d_down = z(E, I, H, dt=torch.float32), z(E, H, I, dt=torch.float32)
    moe.grouped_gemm_dgrad(dy, down, off, da, status=status)
    moe.grouped_gemm_wgrad(dy, a, off, d_down, status=status)
    dh = (da.float() * 2 * torch.relu(h.float())).to(bf)
    moe.grouped_gemm_dgrad(dh, up, off, dxs, status=status)
    moe.grouped_gemm_wgrad(dh, xs, off, d_up, status=status)
    assert int(status.item()) == 0

    o = off.tolist()
    assert o[0] == 0 and o[-1] == R and o[4] == o[3]
    for e in range(E):
        s = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            assert (d_up[e] == 0).all() and (d_down[e] == 0).all()
            continue
        X, U, D, G = (t.double() for t in (xs[s], up[e], down[e], dy[s]))
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        n = lambda t: torch.zeros_like(t)  # noqa: E731
        H0, eh0 = product(X, n(X), U.T, n(U.T))
        A = H0.clamp(min=0) ** 2
        ea = rounded(A, 2 * H0.clamp(min=0) * eh0 + eh0 * eh0)
        eh = rounded(H0, eh0)
        check(h[s], H0, eh, "up")
        check(a[s], A, ea, "up + relu^2")
        Y, ey = product(A, ea, D.T, n(D.T))
        check(y[s], Y, rounded(Y, ey), "down")
        DA, eda = product(G, n(G), D, n(D))
        eda = rounded(DA, eda)
        check(da[s], DA, eda, "gradient of a")
        DD, edd = product(G.T, n(G.T), A, ea)
        check(d_down[e], DD, edd + 2.0 ** -24 * DD.abs(), "gradient of down")
        relu = H0.clamp(min=0)
        DH = DA * 2 * relu
        edh = rounded(DH, eda * 2 * (relu + eh) + DA.abs() * 2 * eh + zero)
        check(dh[s], DH, edh, "gradient of h")
        DX, edx = product(DH, edh, U, n(U))
        check(dxs[s], DX, rounded(DX, edx), "gradient of x")
        DU, edu = product(DH.T, edh.T, X, n(X))
        check(d_up[e], DU, edu + 2.0 ** -24 * DU.abs(), "gradient of up")


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def nvfp4(E, N, K, gen):
    w = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(32, 64, (E, N, K // 16), dtype=torch.uint8, device="cuda", generator=gen)
    s2 = torch.rand(E, device="cuda", generator=gen) * 0.02 + 0.01
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    v = torch.stack((table[(w & 15).long()], table[(w >> 4).long()]), -1).flatten(-2)
    v = v * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * s2.double().view(E, 1, 1)
    return (w, s, s2), v


def test_decode_step_on_nvfp4_experts_with_the_layers_routing():
    shape = WORKLOADS["tiny"]
    inp = make_inputs(shape, T=4)
    layer = moe.MoELayer.from_inputs(inp, max_tokens=16)
    T, k, E, H, I = 4, shape.k, shape.E, shape.H, shape.I
    gen = torch.Generator(device="cuda").manual_seed(22)
    (uw, us, u2), U = nvfp4(E, I, H, gen)
    (dw, ds, d2), D = nvfp4(E, H, I, gen)
    hidden = torch.from_numpy(inp.hidden[:T].view(np.int16).copy()).cuda().view(torch.bfloat16)
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    wts = torch.zeros(T, k, device="cuda")
    a = torch.zeros(T, k, I, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(T, k, H, dtype=torch.bfloat16, device="cuda")

    def step():
        layer.route(hidden, idx, wts)
        moe.nvfp4_gemv(hidden, idx, uw, us, u2, a, relu2=True)
        moe.nvfp4_gemv(a, idx, dw, ds, d2, y)
    try:
        step()
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for turn in range(3):
            hidden.copy_(torch.randn(T, H, device="cuda", generator=gen))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for t in range(T):
                for j in range(k):
                    e = int(idx[t, j])
                    x = hidden[t].double()
                    # the sums' and the digits' part (see test_nvfp4_gemv), then relu^2
                    mag, top = U[e].abs() @ x.abs(), x.abs().max()
                    eh = (H + 8) * 3 * SUM * mag + U[e].abs().sum(1) * top * 2.0 ** -22
                    h0 = U[e] @ x
                    A = h0.clamp(min=0) ** 2
                    ea = rounded(A, 2 * h0.clamp(min=0) * eh + eh * eh + A * 2.0 ** -24)
                    check(a[t, j], A, ea, ("up", turn, t, j))
                    # the down projection of what the up projection left
                    x = a[t, j].double()
                    Y = D[e] @ x
                    ey = (I + 8) * 3 * SUM * (D[e].abs() @ x.abs()) + (
                        D[e].abs().sum(1) * x.abs().max() * 2.0 ** -22) + Y.abs() * 2.0 ** -24
                    check(y[t, j], Y, rounded(Y, ey), ("down", turn, t, j))
        graph.reset()
    finally:
        torch.cuda.synchronize()
        layer.close()
