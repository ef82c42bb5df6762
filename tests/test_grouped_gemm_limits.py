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


def positive(shape, dtype, gen):
    return (torch.rand(*shape, device="cuda", generator=gen) * 0.5 + 0.5).mul_(2.0 ** -4).to(dtype)


def check_long_sums(got, ref, q, piece):
    """Sums of q positive products in pieces of `piece`.  A step of 16 products is added in four parts at
    most, each truncated by less than 2^-23 of the running sum, which is half of the piece's on average
    (2 % more for its spread): piece / 16 * 4 * 2^-23 * 0.51 of the result.  Each joining of pieces rounds
    by 2^-24 of the sum so far, half of the result on average.  Rounding to the type adds at most eps / 2.
    (The errors' mean has no smaller bound: sums of q like terms lie within about q^-1/2 of each other,
    576 +- 0.7 for 262221 products, where BF16's step is 4, so that all round the same way.)"""
    eps = torch.finfo(got.dtype).eps / 2
    lost = piece / 16 * 4 * 2.0 ** -23 * 0.51 + q / piece * 2.0 ** -24 * 0.51
    err = (got.double() - ref) / ref
    assert float(err.abs().max()) <= lost + eps * (1 + lost)


@pytest.mark.parametrize("out", (torch.float16, BF16, torch.float32))
@pytest.mark.parametrize("rows,K,N", ((1 << 20, 64, 72), ((1 << 18) + 77, 136, 64), (8192, 128, 64), (8193, 64, 128),
                                      (16384 + 64, 128, 128), (20000, 2048, 2560)))
def test_long_weight_gradients_of_one_sign(rows, K, N, out):
    gen = torch.Generator(device="cuda").manual_seed(6)
    dt = BF16 if out == BF16 else torch.float16
    x, dy = positive((rows + 40, K), dt, gen), positive((rows + 40, N), dt, gen)
    dw = torch.full((3, N, K), 7.0, dtype=out, device="cuda")
    moe.grouped_gemm_wgrad(dy, x, offsets(0, 40, 40, rows + 40), dw)
    ref = dy[40:].double().T @ x[40:].double()
    check_long_sums(dw[2], ref, rows, 768 if out == torch.float32 else 8192)
    check_long_sums(dw[0], dy[:40].double().T @ x[:40].double(), 40, 40)
    assert (dw[1] == 0).all()
    # random signs: the running sum is the result's size at most, the losses' signs change with it
    x *= torch.randint(0, 2, x.shape, device="cuda", generator=gen) * 2 - 1
    moe.grouped_gemm_wgrad(dy, x, offsets(0, 40, 40, rows + 40), dw)
    ref = dy[40:].double().T @ x[40:].double()
    assert (dw[2].double() - ref).norm() <= (4e-5 + torch.finfo(out).eps / 2) * ref.norm()


@pytest.mark.parametrize("mode", ("fwd", "dgrad"))
@pytest.mark.parametrize("dtype", (torch.float16, BF16))
@pytest.mark.parametrize("counts,q,other", (([40, 0, 1], 131072, 72), ([9], 8193, 64), ([300, 1], 32768 + 8, 64),
                                            ([120] * 4, 16392, 3840), ([1280], 20000, 4096)))
def test_long_contractions_of_one_sign(counts, q, other, dtype, mode):
    gen = torch.Generator(device="cuda").manual_seed(7)
    E, rows = len(counts), sum(counts)
    off = [sum(counts[:e]) for e in range(E + 1)]
    a = positive((rows, q + 7 & ~7), dtype, gen)[:, :q]
    w = positive((E, other, q + 7 & ~7) if mode == "fwd" else (E, q, other), dtype, gen)
    w = w[..., :q] if mode == "fwd" else w
    y = torch.full((rows, other), 7.0, dtype=dtype, device="cuda")
    (moe.grouped_gemm if mode == "fwd" else moe.grouped_gemm_dgrad)(a, w, offsets(*off), y)
    ref = torch.cat([a[off[e]:off[e + 1]].double() @ (w[e].double().T if mode == "fwd" else w[e].double())
                     for e in range(E)])
    check_long_sums(y, ref, q, min(q, 8192))


@pytest.mark.parametrize("mode", ("fwd", "dgrad", "wgrad"))
@pytest.mark.parametrize("q,other", ((131072, 40), (8192 + 64, 200), (65536, 136)))
def test_widest_contractions_are_exact(q, other, mode):
    # whole numbers -1, 0, 1: every partial sum is a whole number below 2^18, exact in float32
    gen = torch.Generator(device="cuda").manual_seed(8)
    counts, dt = [3, 0, 70, 1], torch.float32 if mode == "wgrad" else BF16
    off = [0, 3, 3, 73, 74]
    if mode == "wgrad":
        off = [0, 5, 5, q + 5, q + 6]
        x, dy = whole((q + 6, other), gen, 1), whole((q + 6, 48), gen, 1)
        got = torch.full((4, 48, other), 7.0, dtype=dt, device="cuda")
        moe.grouped_gemm_wgrad(dy, x, offsets(*off), got)
        want = torch.stack([dy[off[e]:off[e + 1]].double().T @ x[off[e]:off[e + 1]].double() for e in range(4)])
    else:
        a = whole((74, q), gen, 1)
        w = whole((4, other, q) if mode == "fwd" else (4, q, other), gen, 1)
        got = torch.full((74, other), 7.0, dtype=dt, device="cuda")
        (moe.grouped_gemm if mode == "fwd" else moe.grouped_gemm_dgrad)(a, w, offsets(*off), got)
        want = torch.cat([a[off[e]:off[e + 1]].double() @ (w[e].double().T if mode == "fwd" else w[e].double())
                          for e in range(4)])
    want = want.to(dt)
    assert (want != 7.0).double().mean() > 0.9 and (want != 0.0).double().mean() > 0.4
    assert torch.equal(got, want)
