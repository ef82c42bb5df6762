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


@pytest.mark.parametrize("dtype", ("bf16", "fp16"))
@pytest.mark.parametrize("T,K", ((1, 256), (2, 512), (3, 288), (8, 1024), (5, 8192)))
def test_elements_count_in_full_whatever_stands_beside_them(T, K, dtype):
    # identity matrices return the rows: every bit pattern of a finite number, each row over the
    # type's whole range
    gen = torch.Generator(device="cuda").manual_seed(4)
    bits = torch.randint(0, 1 << 16, (T, K), device="cuda", generator=gen).to(torch.int16)
    x = bits.view(DT[dtype])
    x[~x.isfinite()] = 1.0
    x[0, 5], x[0, 6] = torch.finfo(x.dtype).max, torch.finfo(x.dtype).smallest_normal
    w = torch.zeros(2, K, K // 2, dtype=torch.uint8, device="cuda")
    n = torch.arange(K, device="cuda")
    w[:, n, n // 2] = torch.where(n % 2 == 0, 0x02, 0x20).to(torch.uint8)
    idx = torch.arange(T, dtype=torch.int32, device="cuda").remainder(2).view(T, 1)
    y = torch.full((T, 1, K), 7.0, dtype=x.dtype, device="cuda")
    moe.nvfp4_gemv(x, idx, w, ones(2, K, K // 16), torch.ones(2, device="cuda"), y)
    assert torch.equal(y[:, 0] + 0.0, x + 0.0)


@pytest.mark.parametrize("dtype,top,rest", (("fp16", 60000.0, 0.1), ("fp16", 600.0, 0.1), ("fp16", 60000.0, 1e-5),
                                            ("bf16", 2.0 ** 20, 1.37), ("bf16", 2.0 ** 60, 1.37),
                                            ("bf16", 3e38, 1e-30), ("bf16", 1e-30, 1e-38)))
def test_outliers_at_weights_of_zero(dtype, top, rest):
    # The rows' digits are exact.  Balanced base-8 digits' magnitudes, times their places, add up to
    # less than 4 |X| (a 1 before digits of -4: 11 / 3).  Each of the K products of a digit is exact,
    # each float32 addition off by at most a unit in the last place, and joining sixteen sums adds
    # sixteen: (K + 16) * 2^-23 * 4 sum |w x|, in which the outliers have no part.
    gen = torch.Generator(device="cuda").manual_seed(5)
    E, N, K, T = 3, 72, 256, 4
    w = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    w[:, :, 0] &= 0xF0
    w[:, :, 100] &= 0x0F
    x = (torch.randn(T, K, device="cuda", generator=gen) * rest).to(DT[dtype])
    x[:, 0], x[:, 201] = top, -top
    idx = torch.tensor([[0, 1], [1, 2], [0, 2], [0, 0]], dtype=torch.int32, device="cuda")
    y = torch.full((T, 2, N), 7.0, dtype=x.dtype, device="cuda")
    moe.nvfp4_gemv(x, idx, w, ones(E, N, K // 16), torch.ones(E, device="cuda"), y)
    f = torch.finfo(x.dtype)
    for t in range(T):
        for j in range(2):
            W, v = values(w)[int(idx[t, j])], x[t].double()
            ref, tol = W @ v, (K + 16) * 2.0 ** -23 * 4 * (W.abs() @ v.abs())
            tol = tol + (ref.abs() + tol) * (f.eps / 2 + 2.0 ** -24) + f.smallest_normal * f.eps / 2
            assert ((y[t, j].double() - ref).abs() <= tol).all(), (t, j)


@pytest.mark.parametrize("K", (2688, 5888, 8192))
@pytest.mark.parametrize("T,k,E", ((1, 2, 4), (2, 2, 4), (3, 2, 20), (30, 2, 8)))
def test_long_sums_of_whole_numbers_are_exact(T, k, E, K):
    # sums of at most 8192 products of magnitude 6 * 8: with the digits' factor 4 below 2^24 halves
    # in every order, so each output is the exact sum, rounded once
    gen = torch.Generator(device="cuda").manual_seed(K)
    N = 150
    w = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.tensor([0x38, 0x30], dtype=torch.uint8, device="cuda")[
        torch.randint(0, 2, (E, N, K // 16), device="cuda", generator=gen)]  # 1 or 1/2
    x = torch.randint(-8, 9, (T, K), device="cuda", generator=gen).to(torch.bfloat16)
    idx = torch.randint(0, E, (T, k), device="cuda", generator=gen).to(torch.int32)
    y = torch.full((T, k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.nvfp4_gemv(x, idx, w, s, torch.ones(E, device="cuda"), y)
    W = values(w) * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    for t in range(T):
        assert torch.equal(y[t] + 0.0, (W[idx[t].long()] @ x[t].double()).to(torch.bfloat16) + 0.0)
