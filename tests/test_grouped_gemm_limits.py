"""The ragged grouped products at the ends of their documented ranges: calls that last, offsets that
fall, the longest contractions.  Operands are small whole numbers wherever that makes the result exact.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA device", allow_module_level=True)

import mixture_experts_ffn_rmsnorm_b200 as moe  # noqa: E402

BF16 = torch.bfloat16


def offsets(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def test_weight_gradient_that_lasts_before_its_first_tail():
    # 3.5e15 operations, three seconds, in a group of whole 16-row steps before a group of five rows:
    # longer than the limit of a wait on the device, a second.  Every element is exact: 128 rows of
    # the large group are not zero and hold 1, 2 or -1, and the five rows hold -2 to 2.
    K, big, small = 81920, 262128, 5
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(1)
    b = torch.tensor([1.0, 2.0, -1.0], device="cuda")[torch.randint(0, 3, (K,), device="cuda", generator=gen)]
    x = torch.zeros(big + small, K, dtype=BF16, device="cuda")
    x[0:big:2048] = b.to(BF16)
    x[big:] = torch.randint(-2, 3, (small, K), device="cuda", generator=gen).to(BF16)
    dw = torch.full((2, K, K), 7.0, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.grouped_gemm_wgrad(x, x, offsets(0, big, big + small), dw, status=status)
    assert int(status.item()) == 0
    for a in range(0, K, 8192):
        assert torch.equal(dw[0, a:a + 8192].float(), 128 * b[a:a + 8192, None] * b)
        t = x[big:].float()
        assert torch.equal(dw[1, a:a + 8192].float(), t[:, a:a + 8192].T @ t)
