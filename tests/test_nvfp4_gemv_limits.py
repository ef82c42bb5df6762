"""moe_nvfp4_gemv at the ends of its documented ranges: launches with idle CTAs, rows of any range,
the longest sums.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA device", allow_module_level=True)

import mixture_experts_ffn_rmsnorm_b200 as moe  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def values(w):
    """E2M1 values [.., K] of packed codes [.., K / 2], in 64 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    return torch.stack((table[(w & 15).long()], table[(w >> 4).long()]), -1).flatten(-2)


def ones(*shape):
    return torch.full(shape, 0x38, dtype=torch.uint8, device="cuda")


def test_launches_with_idle_ctas():
    # repeated and invalid ids leave most of the launch's CTAs without work; calls follow one another
    # so that their starts and ends overlap
    gen = torch.Generator(device="cuda").manual_seed(1)
    E, N, K, T, k = 3, 40, 96, 100, 4
    w = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    x = torch.randint(-2, 3, (T, K), device="cuda", generator=gen).to(torch.bfloat16)
    W = values(w)
    for ids in ([-1] * 4, [2, -1, 7, -1], [1, 1, 1, 1]):
        idx = torch.tensor(ids, dtype=torch.int32, device="cuda").repeat(T, 1)
        ys = [torch.full((T, k, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
        for y in ys:
            moe.nvfp4_gemv(x, idx, w, ones(E, N, K // 16), torch.ones(E, device="cuda"), y)
        for j, e in enumerate(ids):
            want = (x.double() @ W[e].T).to(torch.bfloat16) if 0 <= e < E else torch.zeros_like(ys[0][:, j])
            assert all(torch.equal(y[:, j] + 0.0, want + 0.0) for y in ys)


@pytest.mark.parametrize("dtype", ("bf16", "fp16"))
def test_infinite_and_nan_factors_follow_the_formula(dtype):
    # s2 times a sum that is infinite, zero, finite or NaN, in the order of the formula
    inf, nan = float("inf"), float("nan")
    E, N, K = 4, 16, 32
    w = torch.full((E, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # ones
    w[:, 3:6] = 0xAA  # -1
    w[:, 6:9] = 0x00
    s2 = torch.tensor([inf, -inf, nan, 0.0], device="cuda")
    x = torch.zeros(5, K, dtype=DT[dtype], device="cuda")
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = inf, -inf, 2.0, nan
    idx = torch.arange(E, dtype=torch.int32, device="cuda").repeat(5, 1)
    y = torch.full((5, E, N), 7.0, dtype=DT[dtype], device="cuda")
    moe.nvfp4_gemv(x, idx, w, ones(E, N, K // 16), s2, y)
    for t in range(5):
        # one non-zero element at most: its product with the weight, or 0
        k = min(t, 3)
        want = (x[t, k].double() * values(w)[:, :, k]) * s2.double().view(E, 1)
        torch.testing.assert_close(y[t].double(), want, rtol=0, atol=0, equal_nan=True)
