"""moe_nvfp4_gemv against its definition in 64 bits.

Tolerances.  Weights (E2M1 times unsigned E4M3) are exact.  A token element is
written as a whole number X of units 2^-s with |X| <= 2^22 and its row's largest at
2^21 or above, so it is off by at most half a unit: 2^-22 of the row's largest, times
the sum of the weights' magnitudes.  X has digits -4..3 to base 8 whose magnitudes add
up to at most 3 |X|, and a product of a weight and a digit is exact in float32.  A
float32 sum of K products, in any order and with every addition off by at most one
unit in the last place (2^-23 of the partial sum, truncation allowed), is off by at
most K * 2^-23 of the sum of their magnitudes; joining eight digits' sums adds eight
such steps: together (K + 8) * 2^-23 * 3 S, S the sum of |w x|.  Scaling the sum to
float32 and rounding the result to its type add half a step each (2^-24 and eps / 2 of
the value, and half the smallest subnormal of the type); relu^2 of a value off by d is
off by at most 2 |v| d + d^2.
"""
from concurrent.futures import ThreadPoolExecutor

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA device", allow_module_level=True)

import mixture_experts_ffn_rmsnorm_b200 as moe  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BAD_INDEX_BIT = 2


def weights(E, N, K, gen):
    """Codes uniform over all 16, scales over all finite unsigned E4M3 values (subnormals among them)."""
    w = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(0, 127, (E, N, K // 16), dtype=torch.uint8, device="cuda", generator=gen)
    s2 = torch.rand(E, device="cuda", generator=gen) * 1e-3
    return w, s, s2


def dense(w, s, s2, e):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    c = torch.stack((table[(w[e] & 15).long()], table[(w[e] >> 4).long()]), -1).flatten(-2)
    return c * s[e].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * s2[e].double()


def expected(x, idx, w, s, s2, relu2, dtype):
    T, k = idx.shape
    N, K = w.shape[1], w.shape[2] * 2
    ref = torch.zeros(T, k, N, dtype=torch.float64, device="cuda")
    d = torch.zeros_like(ref)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if not 0 <= e < w.shape[0]:
                continue
            W, v = dense(w, s, s2, e), (x[t, j] if x.dim() == 3 else x[t]).double()
            ref[t, j] = W @ v
            d[t, j] = (K + 8) * 2.0 ** -23 * 3 * (W.abs() @ v.abs()) + (
                W.abs().sum(1) * v.abs().max() * 2.0 ** -22)
    d = d + ref.abs() * 2.0 ** -24
    if relu2:
        d = 2 * ref.clamp(min=0) * d + d * d
        ref = ref.clamp(min=0) ** 2
    f = torch.finfo(dtype)
    return ref, d + (ref.abs() + d) * f.eps / 2 + f.smallest_normal * f.eps / 2


def check(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).nan_to_num(nan=1e30).max()),
                           bad.nonzero()[:4].tolist())


def run(T, k, E, N, K, dtype="bf16", per_slot=False, relu2=False, idx=None, seed=0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    w, s, s2 = weights(E, N, K, gen)
    shape = (T, k, K + pad) if per_slot else (T, K + pad)
    x = torch.randn(*shape, device="cuda", generator=gen).to(dt)[..., :K]
    if idx is None:
        idx = torch.rand(T, E, device="cuda", generator=gen).topk(k, dim=1).indices.to(torch.int32)
    y = torch.full((T, k, N + pad), 7.0, dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, s2, y[..., :N], relu2=relu2, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert (y[..., N:] == 7.0).all()
    check(y[..., :N], *expected(x, idx, w, s, s2, relu2, dt))
    return y


@pytest.mark.parametrize("dtype", ("bf16", "fp16"))
@pytest.mark.parametrize("per_slot", (False, True))
@pytest.mark.parametrize("T,k", ((1, 1), (1, 6), (2, 2), (3, 4), (5, 2), (8, 6), (9, 3), (17, 1), (40, 2)))
def test_tokens(T, k, per_slot, dtype):
    run(T, k, E=12, N=48, K=160, dtype=dtype, per_slot=per_slot, relu2=T % 2 == 0, seed=T)


@pytest.mark.parametrize("K", (32, 64, 96, 128, 224, 256, 416, 1856, 2688, 5888, 6144, 8192))
@pytest.mark.parametrize("N", (1, 15, 16, 17, 200))
def test_widths(N, K):
    # E * N * K / 16 is no multiple of 16 for odd N: the last scales take their own way
    run(3, 2, E=3, N=N, K=K, seed=K + N)
    run(8, 1, E=1, N=N, K=K, dtype="fp16", seed=K + N)


def test_widest_outputs():
    run(3, 2, E=4, N=131072, K=32)


@pytest.mark.parametrize("lead,at", ((70, 1), (67, 3), (64, 2)))
def test_outputs_off_16_byte_boundaries(lead, at):
    gen = torch.Generator(device="cuda").manual_seed(8)
    T, k, E, N, K = 3, 2, 5, 64, 96
    w, s, s2 = weights(E, N, K, gen)
    x = torch.randn(T, K, device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.rand(T, E, device="cuda", generator=gen).topk(k, dim=1).indices.to(torch.int32)
    store = torch.full((T * k * lead + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = store[at:at + T * k * lead].view(T, k, lead)[..., :N]
    moe.nvfp4_gemv(x, idx, w, s, s2, y)
    check(y, *expected(x, idx, w, s, s2, False, y.dtype))
    y.fill_(7.0)
    assert (store == 7.0).all()


def test_beside_the_grouped_products_on_other_streams():
    # four streams at once, every result the lone call's bit by bit
    gen = torch.Generator(device="cuda").manual_seed(9)
    E, N, K, T, k = 12, 200, 256, 6, 4
    w, s, s2 = weights(E, N, K, gen)
    x = torch.randn(T, K, device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.rand(T, E, device="cuda", generator=gen).topk(k, dim=1).indices.to(torch.int32)
    rows = 900
    off = torch.tensor([0, 10, 10, 300] + [500] * 8 + [rows], dtype=torch.int32, device="cuda")
    xr = torch.randn(rows, K, device="cuda", generator=gen).to(torch.bfloat16)
    dy = torch.randn(rows, N, device="cuda", generator=gen).to(torch.bfloat16)
    wd = torch.randn(E, N, K, device="cuda", generator=gen).to(torch.bfloat16)

    def outputs():
        z = lambda *sh, dt=torch.bfloat16: torch.zeros(*sh, dtype=dt, device="cuda")  # noqa: E731
        return [z(T, k, N), z(rows, N), z(rows, K), z(E, N, K, dt=torch.float32)]

    calls = [lambda o, st: moe.nvfp4_gemv(x, idx, w, s, s2, o[0], stream=st),
             lambda o, st: moe.grouped_gemm(xr, wd, off, o[1], stream=st),
             lambda o, st: moe.grouped_gemm_dgrad(dy, wd, off, o[2], stream=st),
             lambda o, st: moe.grouped_gemm_wgrad(dy, xr, off, o[3], accumulate=True, stream=st)]
    alone = outputs()
    for c in calls:
        c(alone, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    many = [outputs() for _ in range(10)]
    torch.cuda.synchronize()
    for out in many:
        for c, st in zip(calls, streams):
            c(out, st)
    torch.cuda.synchronize()
    for out in many:
        assert all(torch.equal(a, b) for a, b in zip(alone, out))


def test_one_expert_for_all_rows():
    idx = torch.full((30, 2), 4, dtype=torch.int32, device="cuda")
    run(30, 2, E=5, N=40, K=256, idx=idx, per_slot=True)
    run(30, 2, E=5, N=40, K=256, idx=idx)


def test_most_rows_and_experts():
    run(64, 16, E=256, N=24, K=64)


def test_strides():
    run(4, 3, E=6, N=33, K=96, pad=8, per_slot=True)
    run(4, 3, E=6, N=33, K=96, pad=8)


def test_ids_out_of_range_give_zero_rows():
    gen = torch.Generator(device="cuda").manual_seed(1)
    w, s, s2 = weights(4, 20, 64, gen)
    x = torch.randn(3, 64, device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.tensor([[0, -1], [4, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    y = torch.full((3, 2, 20), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, s2, y, status=status)
    assert int(status.item()) == BAD_INDEX_BIT
    check(y, *expected(x, idx, w, s, s2, False, y.dtype))
    moe.nvfp4_gemv(x, idx.fill_(-1), w, s, s2, y)
    assert (y == 0).all()


def test_every_code_and_scale():
    # a single 1 in the token reads one weight: 16 codes x every finite scale, exactly; the sign
    # bit of a scale is ignored
    codes = torch.arange(16, dtype=torch.uint8, device="cuda")
    scales = torch.tensor([b for b in range(256) if b & 0x7F != 0x7F], dtype=torch.uint8, device="cuda")
    N, K = scales.numel(), 64
    w = torch.zeros(16, N, K // 2, dtype=torch.uint8, device="cuda")
    w[:, :, 18] = (codes << 4).view(16, 1)  # k = 37
    s = scales.view(1, N, 1).expand(16, N, K // 16).contiguous()
    s2 = torch.ones(16, device="cuda")
    x = torch.zeros(1, K, dtype=torch.float16, device="cuda")
    x[0, 37] = 1.0
    idx = torch.arange(16, dtype=torch.int32, device="cuda").view(1, 16)
    y = torch.zeros(1, 16, N, dtype=torch.float16, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, s2, y)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    ref = table.view(16, 1) * scales.view(torch.float8_e4m3fn).double().abs().view(1, N)
    assert torch.equal(y[0].double(), ref + 0.0)


@pytest.mark.parametrize("scale", (1e-38, 1e-30, 1.0, 1e30, 3e38))
def test_range_of_bf16_rows(scale):
    # rows whose elements span 2^40 around any magnitude: each row has a scale of its own
    gen = torch.Generator(device="cuda").manual_seed(7)
    E, N, K = 2, 32, 256
    w, s, s2 = weights(E, N, K, gen)
    s2 = s2.clamp(max=1.0 / max(scale * 1e3, 1e-30)) if scale > 1 else s2
    x = torch.randn(4, K, device="cuda", generator=gen).clamp(-1, 1)
    x = x * torch.exp2(-torch.randint(0, 40, x.shape, device="cuda", generator=gen).float())
    x = (x.double() * scale * torch.tensor([1.0, 0.5, 1e-3, 0.25], device="cuda").view(4, 1)).to(torch.bfloat16)
    idx = torch.tensor([[0], [1], [0], [0]], dtype=torch.int32, device="cuda")
    y = torch.zeros(4, 1, N, dtype=torch.bfloat16, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, s2, y)
    check(y, *expected(x, idx, w, s, s2, False, y.dtype))


def test_nonfinite_tokens_and_scales():
    gen = torch.Generator(device="cuda").manual_seed(8)
    E, N, K = 2, 32, 128
    w = torch.full((E, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # ones
    s = torch.full((E, N, K // 16), 0x38, dtype=torch.uint8, device="cuda")  # ones
    s2 = torch.ones(E, device="cuda")
    for dt in (torch.bfloat16, torch.float16):
        x = torch.randn(4, K, device="cuda", generator=gen).to(dt)
        x[1, 3] = float("inf")
        x[1, 4] = -60000.0  # finite: the row's sum stays +inf
        x[2, 5] = float("nan")
        idx = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
        y = torch.zeros(4, 1, N, dtype=dt, device="cuda")
        moe.nvfp4_gemv(x, idx, w, s, s2, y)
        assert torch.isposinf(y[1]).all() and y[2].isnan().all()
        assert y[[0, 3]].isfinite().all()
    s[0, 7, 2] = 0x7F  # NaN
    y = torch.zeros(4, 1, N, dtype=dt, device="cuda")
    moe.nvfp4_gemv(torch.ones(4, K, dtype=dt, device="cuda"), idx, w, s, s2, y, relu2=True)
    bad = y.isnan()
    assert bad[:, 0, 7].all() and int(bad.sum()) == 4


def test_bf16_infinity_beside_large_finite_values():
    # 1e30 lies far above FP16's range: it must not turn into an infinity of the other sign
    w = torch.full((1, 16, 16), 0x22, dtype=torch.uint8, device="cuda")
    s = torch.full((1, 16, 2), 0x38, dtype=torch.uint8, device="cuda")
    x = torch.zeros(1, 32, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[0, 1] = float("inf"), -1e30
    idx = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    y = torch.zeros(1, 1, 16, dtype=torch.bfloat16, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, torch.ones(1, device="cuda"), y)
    assert torch.isposinf(y).all()


def test_no_tokens():
    z = lambda *sh, dt=torch.bfloat16: torch.zeros(*sh, dtype=dt, device="cuda")  # noqa: E731
    moe.nvfp4_gemv(z(0, 64), z(0, 2, dt=torch.int32), z(3, 8, 32, dt=torch.uint8),
                   z(3, 8, 4, dt=torch.uint8), z(3, dt=torch.float32), z(0, 2, 8))


def test_captured_replayed_and_deterministic():
    gen = torch.Generator(device="cuda").manual_seed(4)
    E, N, K, T, k = 16, 100, 320, 4, 3
    w, s, s2 = weights(E, N, K, gen)
    x = torch.randn(T, K, device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    y = torch.zeros(T, k, N, dtype=torch.bfloat16, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, s2, y)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        moe.nvfp4_gemv(x, idx, w, s, s2, y)
    x.copy_(torch.randn(T, K, device="cuda", generator=gen))
    idx.copy_(torch.rand(T, E, device="cuda", generator=gen).topk(k, dim=1).indices)
    torch.cuda.synchronize()
    out = []
    for _ in range(3):
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        out.append(y.clone())
    check(out[0], *expected(x, idx, w, s, s2, False, y.dtype))
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    graph.reset()


def test_first_call_of_a_thread():
    # a host thread that has made no CUDA call yet, and one beside it
    gen = torch.Generator(device="cuda").manual_seed(5)
    E, N, K, T, k = 16, 100, 320, 4, 3
    w, s, s2 = weights(E, N, K, gen)
    x = torch.randn(T, K, device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.rand(T, E, device="cuda", generator=gen).topk(k, dim=1).indices.to(torch.int32)
    ys = torch.zeros(3, T, k, N, dtype=torch.bfloat16, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, s2, ys[2])
    check(ys[2], *expected(x, idx, w, s, s2, False, ys.dtype))
    torch.cuda.synchronize()
    with ThreadPoolExecutor(2) as pool:
        for f in [pool.submit(moe.nvfp4_gemv, x, idx, w, s, s2, ys[i]) for i in range(2)]:
            f.result()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[2]) and torch.equal(ys[1], ys[2])


def test_refusals():
    z = lambda *sh, dt=torch.bfloat16: torch.zeros(*sh, dtype=dt, device="cuda")  # noqa: E731
    x, idx, w = z(2, 64), z(2, 3, dt=torch.int32), z(4, 24, 32, dt=torch.uint8)
    s, s2, y = z(4, 24, 4, dt=torch.uint8), z(4, dt=torch.float32), z(2, 3, 24)

    def refused(code, *a):
        with pytest.raises(moe.MoEError) as ei:
            moe.nvfp4_gemv(*a)
        assert ei.value.status == code

    refused(1, z(2, 96), idx, w, s, s2, y)
    refused(1, x, idx.long(), w, s, s2, y)
    refused(1, x, idx, w.to(torch.int8), s, s2, y)
    refused(1, x, idx, w, s[:, :, :3].contiguous(), s2, y)
    refused(1, x, idx, w, s, s2[:3], y)
    refused(1, x, idx, w, s, s2, z(2, 3, 25))
    refused(1, x.float(), idx, w, s, s2, y.float())
    refused(1, x, idx, w, s, s2, y.half())
    refused(1, z(2, 48), idx, z(4, 24, 24, dt=torch.uint8), z(4, 24, 3, dt=torch.uint8), s2, y)
    refused(1, z(2, 66)[:, :64], idx, w, s, s2, y)
    refused(3, z(2, 72)[:, 4:68], idx, w, s, s2, y)
    refused(4, z(400, 64), z(400, 3, dt=torch.int32), w, s, s2, z(400, 3, 24))
    refused(7, x.cpu(), idx, w, s, s2, y)
    torch.cuda.synchronize()
