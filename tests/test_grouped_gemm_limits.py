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


def whole(shape, gen, top=3):
    return torch.randint(-top, top + 1, shape, device="cuda", generator=gen).to(BF16)


def owned(off, rows):
    """(first, last + 1) of the rows whose outputs each group writes; None where it counts as empty."""
    out = []
    for e, (a, b) in enumerate(zip(off, off[1:])):
        ok = 0 <= a <= b <= rows and all(o <= a or o > rows for o in off[:e])
        out.append((a, b) if ok else None)
    return out


@pytest.mark.parametrize("mode", ("fwd", "dgrad"))
@pytest.mark.parametrize("scale", (1, 30))
@pytest.mark.parametrize("off", ([0, 10, 5, 20, 60], [0, 40, 5, 20, 30, 50, 60], [0, 10, 5, 9, 7, 60, 60],
                                 [60, 0, 10, 20, 60], [0, 20, 2 ** 20, 20, 10, 40, 60],
                                 [0, 30, -5, 10, 30, 60]))
def test_rows_that_falling_offsets_give_twice_have_one_owner(off, scale, mode):
    # whole numbers of magnitude at most 64 * 9: exact sums, rounded once; `scale` reaches other tiles
    gen = torch.Generator(device="cuda").manual_seed(2)
    off = [o * scale for o in off]
    rows, E, K, N = 60 * scale, len(off) - 1, 64, 48
    x, w = whole((rows, K if mode == "fwd" else N), gen), whole((E, N, K), gen)
    want = torch.full((rows, N if mode == "fwd" else K), 7.0, dtype=BF16, device="cuda")
    for e, g in enumerate(owned(off, rows)):
        if g:
            m = w[e].float().T if mode == "fwd" else w[e].float()
            want[g[0]:g[1]] = (x[g[0]:g[1]].float() @ m).to(BF16)
    for _ in range(5):
        got = torch.full_like(want, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        (moe.grouped_gemm if mode == "fwd" else moe.grouped_gemm_dgrad)(x, w, offsets(*off), got, status=status)
        assert int(status.item()) == 2
        assert torch.equal(got, want)


def test_weight_gradient_of_rows_that_falling_offsets_give_twice():
    gen = torch.Generator(device="cuda").manual_seed(3)
    off, rows, K, N = [0, 40, 5, 20, 30, 50, 60], 60, 64, 48
    x, dy = whole((rows, K), gen), whole((rows, N), gen)
    dw = torch.full((6, N, K), 7.0, device="cuda")
    moe.grouped_gemm_wgrad(dy, x, offsets(*off), dw)
    for e, (a, b) in enumerate(zip(off, off[1:])):
        want = dy[a:b].float().T @ x[a:b].float() if a <= b else torch.full((N, K), 7.0, device="cuda")
        assert torch.equal(dw[e], want)
