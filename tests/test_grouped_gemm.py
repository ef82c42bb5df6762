"""The ragged grouped products (moe_grouped_gemm and its two gradients) against
the definition in 64 bits, group by group.

Tolerances.  Operands are 16-bit, so a product of two is exact in float32
(22 significant bits at most).  A float32 sum of q products, in any order and
with every addition off by at most one unit in the last place (2^-23 of the
partial sum, truncation allowed), differs from the exact one by at most
d = q * 2^-23 * S, where S is the sum of the products' magnitudes.  relu^2
of a sum off by d is off by at most 2 |s| d + d^2.  One rounding to the output
type adds half a step: eps / 2 of the value (plus half the smallest subnormal).
"""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA device", allow_module_level=True)

import mixture_experts_ffn_rmsnorm_b200 as moe  # noqa: E402

BAD_INDEX_BIT = 2
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def offsets(counts, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(counts)]), dtype=torch.int32,
                        device="cuda")


def padded(shape, dtype, gen, pad=0, std=1.0):
    """A view [..., width] of a tensor whose rows lie (width + pad) rounded up to 8 apart."""
    width = shape[-1]
    wide = (width + pad + 7) // 8 * 8
    t = torch.full((*shape[:-1], wide), float("nan"), device="cuda", dtype=dtype)
    v = t[..., :width]
    v.copy_(torch.randn(*shape, device="cuda", generator=gen) * std)
    return v


def bound(ref, mag, q, dtype, relu2=False):
    d = q * 2.0 ** -23 * mag
    if relu2:
        d = 2 * ref.clamp(min=0) * d + d * d
        ref = ref.clamp(min=0) ** 2
    f = torch.finfo(dtype)
    tiny = torch.finfo(dtype).smallest_normal * f.eps / 2
    return ref, d + (ref.abs() + d) * f.eps / 2 + tiny


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol).nan_to_num(nan=float("inf")).max()),
                           bad.nonzero()[:4].tolist())


def reference(mode, off, E, dy, x, w):
    """(exact result, sum of magnitudes) in 64 bits; zeros outside the groups."""
    o = off.tolist()
    if mode == "fwd":
        ref = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    elif mode == "dgrad":
        ref = torch.zeros(dy.shape[0], w.shape[2], dtype=torch.float64, device="cuda")
    else:
        ref = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for e in range(E):
        a, b = o[e], o[e + 1]
        if b <= a:
            continue
        if mode == "fwd":
            l, r, at = x[a:b].double(), w[e].double().T, slice(a, b)
        elif mode == "dgrad":
            l, r, at = dy[a:b].double(), w[e].double(), slice(a, b)
        else:
            l, r, at = dy[a:b].double().T, x[a:b].double(), e
        ref[at] = l @ r
        mag[at] = l.abs() @ r.abs()
    return ref, mag


def run(mode, counts, K, N, dtype, relu2=False, start=0, tail=0, pad=0, f32=False, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    off = offsets(counts, start)
    rows = start + int(sum(counts)) + tail
    dt = DT[dtype]
    x = padded((rows, K), dt, gen, pad)
    dy = padded((rows, N), dt, gen, pad)
    w = padded((E, N, K), dt, gen, pad, std=K ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # rows that belong to nobody hold NaN: they may not reach any output
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    inside[start:rows - tail] = True
    x[~inside] = float("nan")
    dy[~inside] = float("nan")
    if mode == "fwd":
        out = torch.full((rows, N + pad), 7.0, device="cuda", dtype=dt)[:, :N]
        moe.grouped_gemm(x, w, off, out, relu2=relu2, status=status)
        q = K
    elif mode == "dgrad":
        out = torch.full((rows, K + pad), 7.0, device="cuda", dtype=dt)[:, :K]
        moe.grouped_gemm_dgrad(dy, w, off, out, status=status)
        q = N
    else:
        out = torch.full((E, N, K + pad), 7.0, device="cuda",
                         dtype=torch.float32 if f32 else dt)[..., :K]
        moe.grouped_gemm_wgrad(dy, x, off, out, status=status)
        q = max(counts)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref, mag = reference(mode, off, E, dy, x, w)
    if mode != "wgrad":
        assert (out[~inside] == 7.0).all(), "a row outside every group was written"
        out, ref, mag = out[inside], ref[inside], mag[inside]
    ref, tol = bound(ref, mag, q, out.dtype, relu2)
    check(out, ref, tol, (mode, counts[:8], K, N, dtype))
    return out


MODES = ("fwd", "dgrad", "wgrad")
# few rows a group (the narrow kernel) and many (the pair kernel); groups that are empty, that hold
# one row, that end next to a tile's or a k-block's border, or inside one
FEW = [0, 1, 3, 0, 17, 16, 15, 2, 33, 64, 65, 1]
MANY = [255, 0, 1, 256, 257, 63, 64, 65, 300, 47, 513, 130]


@pytest.mark.parametrize("dtype", ("bf16", "fp16"))
@pytest.mark.parametrize("counts", (FEW, MANY), ids=("few", "many"))
@pytest.mark.parametrize("mode", MODES)
def test_ragged_groups(mode, counts, dtype):
    run(mode, counts, K=256, N=128, dtype=dtype)


@pytest.mark.parametrize("K,N", ((1, 1), (1, 300), (300, 1), (7, 9), (63, 65), (64, 64), (72, 200),
                                 (129, 257), (517, 333), (1000, 96)))
@pytest.mark.parametrize("counts", ([5, 0, 40, 2], [200, 3, 0, 301]), ids=("few", "many"))
@pytest.mark.parametrize("mode", MODES)
def test_odd_widths(mode, counts, K, N):
    run(mode, counts, K=K, N=N, dtype="bf16", seed=K)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("counts", ([1], [0], [0, 0, 1, 0], [700], [2000, 1], [1] * 256, [40] * 256),
                         ids=lambda c: f"{len(c)}x{max(c)}")
def test_group_counts(mode, counts):
    run(mode, counts, K=136, N=72, dtype="fp16")


@pytest.mark.parametrize("dtype", ("bf16", "fp16"))
@pytest.mark.parametrize("K,N", ((1000, 1024), (2040, 1992), (1999, 2001)))
@pytest.mark.parametrize("mode", MODES)
def test_ragged_groups_with_many_tiles(mode, K, N, dtype):
    # enough tiles that the CTA pairs take them, 128 or 256 rows at a time
    run(mode, MANY, K=K, N=N, dtype=dtype, relu2=mode == "fwd", start=3, tail=2)
    if dtype == "bf16":
        run(mode, [700, 0, 90, 1030, 256, 257], K=K, N=N, dtype=dtype, f32=True)


@pytest.mark.parametrize("K,N", ((2040, 1992), (1999, 2001), (64, 4100)))
@pytest.mark.parametrize("mode", ("fwd", "dgrad"))
def test_groups_just_above_256_rows(mode, K, N):
    # groups that fit one wide tile beside groups that do not; neighbouring tiles that fit the
    # accumulators together, and that do not
    for seed, counts in enumerate(([257, 320, 300, 0, 321, 289, 272, 256, 1, 255, 513, 304],
                                   [320] * 12, [257, 255] * 8, [304, 17, 31, 33] + [318] * 9)):
        avg = sum(counts) / len(counts)
        assert 200 < avg <= 320
        run(mode, counts, K=K, N=N, dtype="bf16", relu2=mode == "fwd", start=1, tail=1, seed=seed)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("rows", (1, 130, 700, 5000))
def test_one_group_with_few_and_with_many_tiles(mode, rows):
    # one dense matrix: the same rows as few small, many small and large tiles
    run(mode, [rows], K=384, N=320, dtype="bf16", f32=rows == 700)
    run(mode, [rows], K=2048, N=1536, dtype="fp16")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("counts", ([9, 30, 0, 5], [90, 300, 0, 5]), ids=("few", "many"))
def test_strides_and_rows_outside_the_groups(mode, counts):
    # operands and outputs with padded rows, rows before the first and behind the last group;
    # pad 3 leaves the output's rows unaligned
    run(mode, counts, K=200, N=136, dtype="bf16", start=5, tail=11, pad=24)
    run(mode, counts, K=200, N=136, dtype="bf16", start=1, tail=1, pad=3)


@pytest.mark.parametrize("mode", MODES + ("wgrad_f32",))
@pytest.mark.parametrize("counts", ([3, 0, 40, 1], [300, 0, 70, 513]), ids=("few", "many"))
@pytest.mark.parametrize("width,lead,at", ((130, 140, 1), (257, 260, 2), (261, 261, 0), (64, 67, 3),
                                           (384, 388, 4), (128, 129, 1), (95, 104, 7), (33, 40, 8),
                                           (250, 256, 0), (36, 40, 8)))
def test_outputs_off_16_byte_boundaries(mode, counts, width, lead, at):
    # rows `lead` elements apart that begin `at` elements into the tensor; what lies beside them stays
    gen = torch.Generator(device="cuda").manual_seed(31)
    mode, f32 = mode[:5], mode.endswith("f32")
    K, N = (72, width) if mode == "fwd" else (width, 72)
    E, rows, off = len(counts), sum(counts), offsets(counts)
    x, dy = padded((rows, K), torch.bfloat16, gen), padded((rows, N), torch.bfloat16, gen)
    w = padded((E, N, K), torch.bfloat16, gen)
    shape = (E, N) if mode == "wgrad" else (rows,)
    store = torch.full((int(np.prod(shape)) * lead + 16,), 7.0, device="cuda",
                       dtype=torch.float32 if f32 else torch.bfloat16)
    out = store[at:at + int(np.prod(shape)) * lead].view(*shape, lead)[..., :width]
    if mode == "fwd":
        moe.grouped_gemm(x, w, off, out)
    elif mode == "dgrad":
        moe.grouped_gemm_dgrad(dy, w, off, out)
    else:
        moe.grouped_gemm_wgrad(dy, x, off, out)
    ref, mag = reference(mode, off, E, dy, x, w)
    check(out, *bound(ref, mag, 513 if mode == "wgrad" else 72, out.dtype), (mode, width))
    out.fill_(7.0)
    assert (store == 7.0).all()


@pytest.mark.parametrize("counts", ([10, 0, 3, 50], [400, 0, 77, 1100]), ids=("few", "many"))
def test_fused_relu2(counts):
    run("fwd", counts, K=264, N=192, dtype="bf16", relu2=True)
    run("fwd", counts, K=264, N=190, dtype="fp16", relu2=True)


@pytest.mark.parametrize("counts", ([10, 0, 3, 50], [400, 0, 77, 1100]), ids=("few", "many"))
def test_weight_gradient_in_32_bits_and_accumulated(counts):
    run("wgrad", counts, K=264, N=190, dtype="bf16", f32=True)
    for K, N in ((100, 52), (1300, 1100)):  # single CTAs, CTA pairs
        accumulated(counts, K, N)


def accumulated(counts, K, N):
    gen = torch.Generator(device="cuda").manual_seed(3)
    E, rows = len(counts), sum(counts)
    off = offsets(counts)
    x, dy = padded((rows, K), torch.float16, gen), padded((rows, N), torch.float16, gen)
    dw = torch.randn(E, N, K, device="cuda", generator=gen)
    before = dw.clone()
    moe.grouped_gemm_wgrad(dy, x, off, dw, accumulate=True)
    ref, mag = reference("wgrad", off, E, dy, x, None)
    ref, tol = bound(ref + before.double(), mag + before.double().abs(), max(counts) + 1, dw.dtype)
    check(dw, ref, tol, "accumulate")
    assert torch.equal(dw[1], before[1])  # nothing to add to an empty group


@pytest.mark.parametrize("K", (64, 65))
def test_accumulation_onto_small_and_special_values(K):
    # subnormals, infinities and NaN in the gradient that is added to; a sum of nothing but zeros
    E, N, counts = 3, 40, [900, 5, 0]
    rows, off = sum(counts), offsets(counts)
    x = torch.zeros(rows, (K + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :K]
    dy = torch.ones(rows, N, dtype=torch.bfloat16, device="cuda")
    x[900] = 1.0  # group 1: every sum is 1
    row = torch.tensor([1e-40, -3e-42, float("inf"), -float("inf"), float("nan"), 2.0, -0.5, 1e30])
    dw = row.cuda().repeat(E * N * K // 8 + 1)[:E * N * K].view(E, N, K).clone()
    before = dw.clone()
    moe.grouped_gemm_wgrad(dy, x, off, dw, accumulate=True)
    torch.testing.assert_close(dw[0], before[0], rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(dw[1], before[1] + 1.0, rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(dw[2], before[2], rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("f32_counts", ([900, 65, 1537, 0, 2000], [769] * 6))
def test_accumulation_is_deterministic(f32_counts):
    gen = torch.Generator(device="cuda").manual_seed(41)
    K, N, E, rows, off = 264, 520, len(f32_counts), sum(f32_counts), offsets(f32_counts)
    x, dy = padded((rows, K), torch.bfloat16, gen), padded((rows, N), torch.bfloat16, gen)
    start = torch.randn(E, N, K, device="cuda", generator=gen)
    runs = []
    for _ in range(4):
        dw = start.clone()
        moe.grouped_gemm_wgrad(dy, x, off, dw, accumulate=True)
        moe.grouped_gemm_wgrad(dy, x, off, dw, accumulate=True)
        runs.append(dw)
    assert all(torch.equal(runs[0], r) for r in runs[1:])
    ref, mag = reference("wgrad", off, E, dy, x, None)
    q = 2 * max(f32_counts) + 1
    check(runs[0], *bound(start.double() + 2 * ref, start.double().abs() + 2 * mag, q, dw.dtype), "acc")


@pytest.mark.parametrize("rows,K,N", ((8192, 512, 512), (8191, 2048, 2304), (769, 96, 40)))
def test_long_sums_in_32_bits(rows, K, N):
    # Every addition of a k-step truncates by less than an ulp (2^-23) of the partial sum.  Sums of
    # random signs grow as the square root of their length, so 48 steps lose less than
    # 48 * 2/3 * 2^-23 = 3.9e-6 of the result in the 2-norm; without a fresh start every 768 rows the
    # 512 steps of 8192 rows could lose 4.1e-5 (and lost 9.1e-6).
    gen = torch.Generator(device="cuda").manual_seed(17)
    x, dy = padded((rows, K), torch.bfloat16, gen), padded((rows, N), torch.bfloat16, gen)
    dw = torch.full((1, N, K), 7.0, device="cuda")
    moe.grouped_gemm_wgrad(dy, x, offsets([rows]), dw)
    ref = dy.double().T @ x.double()
    assert (dw[0].double() - ref).norm() <= 3.9e-6 * ref.norm()
    moe.grouped_gemm_wgrad(dy, x, offsets([rows]), dw, accumulate=True)
    assert (dw[0].double() - 2 * ref).norm() <= 3.9e-6 * 2 * ref.norm()
    run("wgrad", [rows - 700, 0, 700], K=K, N=N, dtype="bf16", f32=True)


@pytest.mark.parametrize("f32", (False, True))
@pytest.mark.parametrize("blocks", (1, 2, 4, 5, 6))
def test_tails_of_neighbouring_tiles_in_one_stage(blocks, f32):
    # every group ends inside the same k-block of the ring, tile after tile on each CTA pair
    run("wgrad", [64 * blocks - 3] * 24, K=768, N=1536, dtype="bf16", f32=f32, seed=blocks)


@pytest.mark.parametrize("f32", (False, True))
@pytest.mark.parametrize("K,N", ((264, 520), (72, 56)))
def test_tails_out_of_turn(f32, K, N):
    # groups whose rows end inside a k-block, of one k-block and of more, around the borders of
    # the 768-row pieces of an FP32 sum
    run("wgrad", [1, 65, 767, 769, 129, 785, 833, 193, 897, 1537, 0, 1600, 63], K, N, "bf16",
        f32=f32, tail=9)


@pytest.mark.parametrize("bad", (float("inf"), float("nan")))
@pytest.mark.parametrize("counts", ([10, 7, 3, 50], [400, 13, 77, 110]), ids=("few", "many"))
def test_nonfinite_values_stay_in_their_group(counts, bad):
    gen = torch.Generator(device="cuda").manual_seed(5)
    E, K, N, rows = 4, 136, 72, sum(counts)
    off = offsets(counts)
    x, dy = padded((rows, K), torch.bfloat16, gen), padded((rows, N), torch.bfloat16, gen)
    w = padded((E, N, K), torch.bfloat16, gen)
    a, b = int(off[1]), int(off[2])
    x[a:b], dy[a:b], w[1] = bad, bad, bad
    y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    dx = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    moe.grouped_gemm(x, w, off, y, relu2=True)
    moe.grouped_gemm_dgrad(dy, w, off, dx)
    moe.grouped_gemm_wgrad(dy, x, off, dw)
    for t in (y, dx):
        assert t[:a].isfinite().all() and t[b:].isfinite().all()
        assert not t[a:b].isfinite().any()
    assert dw[[0, 2, 3]].isfinite().all() and not dw[1].isfinite().any()


@pytest.mark.parametrize("rows", (60, 900))
def test_bad_offsets_are_flagged_and_their_groups_left(rows):
    gen = torch.Generator(device="cuda").manual_seed(6)
    E, K, N = 4, 72, 40
    x, dy = padded((rows, K), torch.bfloat16, gen), padded((rows, N), torch.bfloat16, gen)
    w = padded((E, N, K), torch.bfloat16, gen)
    for off_l, good in (([0, 10, 5, 20, rows], (0, 2, 3)), ([0, 10, 20, 30, rows + 1], (0, 1, 2)),
                        ([-1, 10, 20, 30, rows], (1, 2, 3)),
                        ([2 ** 31 - 1, 10, 20, 30, rows], (1, 2, 3))):
        off = torch.tensor(off_l, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((E, N, K), 7.0, dtype=torch.float32, device="cuda")
        moe.grouped_gemm(x, w, off, y, status=status)
        assert int(status.item()) == BAD_INDEX_BIT
        status.zero_()
        moe.grouped_gemm_wgrad(dy, x, off, dw, status=status)
        assert int(status.item()) == BAD_INDEX_BIT
        inside = torch.zeros(rows, dtype=torch.bool)
        for e in range(E):
            a, b = off_l[e], off_l[e + 1]
            if e in good:
                inside[a:b] = True
                ref = dy[a:b].double().T @ x[a:b].double()
                mag = dy[a:b].double().abs().T @ x[a:b].double().abs()
                check(dw[e], *bound(ref, mag, b - a, dw.dtype), off_l)
            else:
                assert (dw[e] == 7.0).all()
        assert (y[~inside.cuda()] == 7.0).all()


def test_no_rows():
    E, K, N = 3, 64, 48
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w, dw = z(E, N, K), torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.grouped_gemm(z(0, K), w, off, z(0, N))
    moe.grouped_gemm_dgrad(z(0, N), w, off, z(0, K))
    moe.grouped_gemm_wgrad(z(0, N), z(0, K), off, dw)
    assert (dw == 0).all()


def test_offsets_past_32_bits():
    # rows 2^21 elements apart: the last ones lie behind element 2^31 of operand and output
    ld, rows, K, N = 1 << 21, 1100, 64, 40
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")[:, :K]
    y = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")[:, :N]
    x.copy_(torch.randn(rows, K, device="cuda", generator=gen))
    w = padded((2, N, K), torch.bfloat16, gen)
    off = offsets([500, 600])
    moe.grouped_gemm(x, w, off, y)
    ref, mag = reference("fwd", off, 2, None, x, w)
    check(y, *bound(ref, mag, K, y.dtype), "far rows")


def test_captured_and_replayed_beside_another_stream():
    # two graphs of the same kernels, replayed on two streams at once, on inputs written after
    # the capture
    gen = torch.Generator(device="cuda").manual_seed(11)
    E, K, N = 6, 264, 200
    sets = []
    for s in range(2):
        counts = [300, 0, 25, 64, 1, 129]
        rows = sum(counts)
        t = dict(off=offsets(counts), x=padded((rows, K), torch.bfloat16, gen),
                 dy=padded((rows, N), torch.bfloat16, gen), w=padded((E, N, K), torch.bfloat16, gen),
                 y=torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"),
                 dx=torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda"),
                 dw=torch.zeros(E, N, K, device="cuda"), stream=torch.cuda.Stream())

        def calls(t=t):
            moe.grouped_gemm(t["x"], t["w"], t["off"], t["y"])
            moe.grouped_gemm_dgrad(t["dy"], t["w"], t["off"], t["dx"])
            moe.grouped_gemm_wgrad(t["dy"], t["x"], t["off"], t["dw"])
        calls()
        torch.cuda.synchronize()
        t["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(t["graph"], stream=t["stream"]):
            calls()
        sets.append(t)
    for t in sets:
        t["x"].copy_(torch.randn(*t["x"].shape, device="cuda", generator=gen))
        t["off"].copy_(offsets([10, 200, 0, 3, 250, 56]))
        for n in ("y", "dx", "dw"):
            t[n].fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(3):
        for t in sets:
            with torch.cuda.stream(t["stream"]):
                t["graph"].replay()
    torch.cuda.synchronize()
    for t in sets:
        for mode, name, q in (("fwd", "y", K), ("dgrad", "dx", N), ("wgrad", "dw", 250)):
            ref, mag = reference(mode, t["off"], E, t["dy"], t["x"], t["w"])
            check(t[name], *bound(ref, mag, q, t[name].dtype), name)
        t["graph"].reset()


def test_streams_that_join_inside_one_capture():
    # forward and weight gradient on two streams forked from the capturing one, the data gradient
    # after the join; each launch has dependencies on other streams
    gen = torch.Generator(device="cuda").manual_seed(21)
    E, K, N = 5, 328, 264
    counts = [700, 3, 0, 64, 257]
    rows = sum(counts)
    off, off0 = offsets(counts), offsets(counts)
    x, dy = padded((rows, K), torch.bfloat16, gen), padded((rows, N), torch.bfloat16, gen)
    w = padded((E, N, K), torch.bfloat16, gen)
    y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    dx = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        off.copy_(off0)
        side.wait_stream(here)
        moe.grouped_gemm(x, w, off, y)
        with torch.cuda.stream(side):
            moe.grouped_gemm_wgrad(dy, x, off, dw)
        here.wait_stream(side)
        moe.grouped_gemm_dgrad(y, w, off, dx)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        off0.copy_(offsets([100, 300, 24, 600, 0]))
        x.copy_(torch.randn(rows, K, device="cuda", generator=gen))
        for t in (y, dx, dw, off):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for mode, out, q in (("fwd", y, K), ("dgrad", dx, N), ("wgrad", dw, 600)):
            ref, mag = reference(mode, off0, E, y if mode == "dgrad" else dy, x, w)
            check(out, *bound(ref, mag, q, out.dtype), (mode, seed))
    graph.reset()


def test_threads_at_once():
    # two host threads, a stream each, the same weights; every result is the lone call's, bit by bit
    gen = torch.Generator(device="cuda").manual_seed(22)
    E, K, N = 6, 512, 328
    counts = [300, 0, 1, 47, 600, 64]
    rows, off = sum(counts), offsets(counts)
    w = padded((E, N, K), torch.bfloat16, gen)
    xs = [padded((rows, K), torch.bfloat16, gen) for _ in range(2)]
    dys = [padded((rows, N), torch.bfloat16, gen) for _ in range(2)]

    def outputs():
        return (torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(E, N, K, device="cuda"))

    def calls(i, out, stream):
        moe.grouped_gemm(xs[i], w, off, out[0], stream=stream)
        moe.grouped_gemm_dgrad(dys[i], w, off, out[1], stream=stream)
        moe.grouped_gemm_wgrad(dys[i], xs[i], off, out[2], stream=stream)

    alone = [outputs() for _ in range(2)]
    for i in range(2):
        calls(i, alone[i], None)
    many = [[outputs() for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream()
        for out in many[i]:
            calls(i, out, stream)
        stream.synchronize()

    with ThreadPoolExecutor(2) as pool:
        for f in [pool.submit(work, i) for i in range(2)]:
            f.result()
    for i in range(2):
        for out in many[i]:
            assert all(torch.equal(a, b) for a, b in zip(alone[i], out))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("K,N", ((131072, 8), (8, 131072)))
def test_widest_matrices(mode, K, N):
    run(mode, [5, 0, 70], K, N, "bf16")


@pytest.mark.parametrize("mode", ("fwd", "dgrad"))
def test_most_rows(mode):
    # 2^24 rows of 8 elements: the largest row numbers, in the last groups
    rows, K, N = 1 << 24, 8, 8
    gen = torch.Generator(device="cuda").manual_seed(23)
    a = torch.randint(-3, 4, (rows, 8), device="cuda", generator=gen).to(torch.bfloat16)
    w = torch.randint(-3, 4, (3, N, K), device="cuda", generator=gen).to(torch.bfloat16)
    off = offsets([rows - 1000, 999, 1])
    out = torch.full((rows, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    (moe.grouped_gemm if mode == "fwd" else moe.grouped_gemm_dgrad)(a, w, off, out)
    # whole numbers of magnitude at most 72: exact in bfloat16
    for e, (lo, hi) in enumerate(((0, rows - 1000), (rows - 1000, rows - 1), (rows - 1, rows))):
        m = w[e].float().T if mode == "fwd" else w[e].float()
        assert torch.equal(out[lo:hi].float(), (a[lo:hi, :, None].float() * m).sum(1)), e


def test_gradients_against_differences():
    # directional derivatives of L = sum(g * y): the products are linear in x and in w, so a
    # difference quotient has no truncation error; what is left is the roundings of both sides,
    # bounded by half a step of every y (times |g|) and of every gradient element (times the step)
    gen = torch.Generator(device="cuda").manual_seed(12)
    counts, K, N = [130, 0, 40, 7], 96, 80
    rows, E = sum(counts), len(counts)
    off = offsets(counts)
    x = torch.randint(-4, 5, (rows, K), device="cuda", generator=gen).to(torch.bfloat16)
    w = torch.randint(-4, 5, (E, N, K), device="cuda", generator=gen).to(torch.bfloat16)
    g = torch.randint(-2, 3, (rows, N), device="cuda", generator=gen).to(torch.bfloat16)
    sx = torch.randint(-1, 2, (rows, K), device="cuda", generator=gen).to(torch.bfloat16)
    sw = torch.randint(-1, 2, (E, N, K), device="cuda", generator=gen).to(torch.bfloat16)

    def loss(x_, w_):
        y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
        moe.grouped_gemm(x_, w_, off, y)
        return (g.double() * y.double()).sum(), (g.double() * y.double()).abs().sum() * 2.0 ** -8

    dx = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(E, N, K, device="cuda")
    moe.grouped_gemm_dgrad(g, w, off, dx)
    moe.grouped_gemm_wgrad(g, x, off, dw)
    base, tol0 = loss(x, w)
    fx, tolx = loss(x + sx, w)  # small whole numbers: the sums x + sx are exact
    assert abs(fx - base - (dx.double() * sx.double()).sum()) <= (
        tol0 + tolx + (dx.double() * sx.double()).abs().sum() * 2.0 ** -8)
    fw, tolw = loss(x, w + sw)
    assert abs(fw - base - (dw.double() * sw.double()).sum()) <= tol0 + tolw


def test_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, w, y, dw = z(8, 64), z(2, 48, 64), z(8, 48), z(2, 48, 64)

    def refused(code, f, *a, **kw):
        with pytest.raises(moe.MoEError) as ei:
            f(*a, **kw)
        assert ei.value.status == code

    refused(1, moe.grouped_gemm, z(8, 72), w, off, y)                     # K differs
    refused(1, moe.grouped_gemm, x, w, off, z(9, 48))                     # rows differ
    refused(1, moe.grouped_gemm, x, w, off[:2], y)                        # off too short
    refused(1, moe.grouped_gemm, x, w, off.long(), y)
    refused(1, moe.grouped_gemm, x, w.half(), off, y)
    refused(1, moe.grouped_gemm, x.float(), w.float(), off, y.float())
    refused(1, moe.grouped_gemm, z(64, 8).T, w, off, y)                   # rows not contiguous
    refused(1, moe.grouped_gemm, z(8, 65)[:, :64], w, off, y)             # 65 elements apart
    refused(1, moe.grouped_gemm, x, z(2, 96, 64)[:, :48], off, y)         # a gap between experts
    refused(3, moe.grouped_gemm, z(8, 80)[:, 4:68], w, off, y)            # off a 16-byte boundary
    refused(1, moe.grouped_gemm_wgrad, y, x, off, dw, accumulate=True)    # 16-bit accumulation
    refused(1, moe.grouped_gemm_wgrad, y, x, off, z(2, 48, 64, dt=torch.float16))
    refused(7, moe.grouped_gemm, x.cpu(), w, off, y)
    refused(7, moe.grouped_gemm_dgrad, y, w, off, x.cpu())
    torch.cuda.synchronize()
