"""What is measured of the handle-free expert operators: their cases, inputs, plain forms and definition.

Four operators work on routed rows (see include/moe_b200.h): the ragged grouped product
``grouped_gemm`` (rows sorted by expert, group boundaries ``off``), its two gradients
``grouped_gemm_dgrad`` and ``grouped_gemm_wgrad``, and ``nvfp4_gemv``, the matrix-vector
products of a few tokens with experts stored in 4 bits (E2M1 values, one E4M3 scale per 16
inputs, one float32 scale per expert).

``run`` makes one pass: the plain form in elementary torch operations, or, with ``own`` set,
the calls a user makes of the package.  Sizes are those of the repository's workloads (tiny,
decode, prefill, latent, skew_fp8) or generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
# E2M1: sign, two exponent bits, one mantissa bit
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _case(op, name=None, **kw):
    c = {"op": op, "T": 1, "E": 1, "k": 1, "K": 64, "N": 64, "dtype": "bf16", "zipf": 0.0, "tail": 0,
         "relu2": False, "out": "same", "per_slot": False}
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # the smallest layer's up projection: nothing but latency
        _case("fwd", "fwd tiny 16 tokens", T=16, E=8, k=2, K=256, N=128, relu2=True),
        # a serving step of eight requests, up projection with its activation: weights streamed for one or two rows each
        _case("fwd", "fwd decode 8 tokens", T=8, E=128, k=6, K=2688, N=1856, relu2=True),
        # a prompt of 1024 tokens, up projection in half precision: 48 rows an expert
        _case("fwd", "fwd prefill 1024 fp16", T=1024, E=128, k=6, K=2688, N=1856, dtype="fp16", relu2=True),
        # the largest batch under a skewed routing, down projection: bound by the tensor cores
        _case("fwd", "fwd skewed 8192 down", T=8192, E=128, k=6, K=1856, N=2688, zipf=1.2),
        # fine-tuning a small model: sizes that fit no tile, rows behind the last group
        _case("dgrad", "dgrad odd 333 fp16", T=333, E=20, k=3, K=517, N=1003, dtype="fp16", tail=7),
        # training the latent layer's down projection
        _case("dgrad", "dgrad latent 4096", T=4096, E=128, k=8, K=2688, N=1024),
        # a small micro-batch: the gradient's own size is the bound
        _case("wgrad", "wgrad prefill 1024", T=1024, E=128, k=6, K=2688, N=1856),
        # training the latent layer's up projection, gradient kept in 32 bits
        _case("wgrad", "wgrad latent 4096 f32", T=4096, E=128, k=8, K=1024, N=2688, out="f32"),
        # the largest batch under a skewed routing, up projection
        _case("wgrad", "wgrad skewed 8192", T=8192, E=128, k=6, K=2688, N=1856, zipf=1.2),
        # one request's next token, up projection with its activation
        _case("gemv", "gemv 1 token up", T=1, E=128, k=6, K=2688, N=1856, relu2=True),
        # the same token's down projection on the latent layer: each slot has a row of its own
        _case("gemv", "gemv 1 token latent down", T=1, E=128, k=8, K=2688, N=1024, per_slot=True),
        # eight requests' down projection in half precision
        _case("gemv", "gemv 8 tokens down fp16", T=8, E=128, k=6, K=1856, N=2688, per_slot=True, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """A case of the ranges above: one token to the largest batch, one expert to 128, widths from 64 to 2688, odd ones among
    them; never more rows, weights or products than the largest listed case has."""
    op = rng.choice(("fwd", "dgrad", "wgrad", "gemv"))
    E = _log(rng, 1, 128)
    k = rng.randint(1, min(E, 8))
    K, N = _log(rng, 64, 2688), _log(rng, 64, 2688)
    dtype = rng.choice(("bf16", "fp16"))
    relu2 = rng.random() < 0.5
    if op == "gemv":
        return _case(op, T=_log(rng, 1, 16), E=E, k=k, K=max(64, K // 32 * 32), N=N, dtype=dtype, relu2=relu2,
                     per_slot=rng.random() < 0.5)
    T = _log(rng, 1, 8192)
    k = max(1, min(k, 6 * 8192 // T))
    while E * N * K > 128 * 2688 * 1856:
        N = N // 2 + 1
    zipf = rng.choice((0.0, 0.0, 0.6, 1.2))
    out = rng.choice(("same", "f32")) if op == "wgrad" and T <= 2048 else "same"
    return _case(op, T=T, E=E, k=k, K=K, N=N, dtype=dtype, zipf=zipf, relu2=relu2 and op == "fwd", out=out,
                 tail=rng.choice((0, 0, 1, 13)))


def _padded(rows, cols, dtype, gen, std):
    """Normal values [..., cols] whose rows start 16 bytes apart: a view of a wider tensor where cols is no multiple of eight."""
    wide = (cols + 7) // 8 * 8
    t = torch.randn(*rows, wide, device="cuda", dtype=dtype, generator=gen)
    return t.mul_(std)[..., :cols]


def _routing(c, gen):
    """top-k experts of each token, distinct: uniform, or with popularity rank^-zipf over a random order of the experts."""
    rank = torch.randperm(c["E"], device="cuda", generator=gen) + 1
    score = -c["zipf"] * torch.log(rank.float())
    u = torch.rand(c["T"], c["E"], device="cuda", generator=gen).clamp_(1e-20, 1.0 - 1e-7)
    return (score - torch.log(-torch.log(u))).topk(c["k"], dim=1).indices.to(torch.int32)


def _quantise(w):
    """NVFP4 of w [E, N, K]: (packed codes [E, N, K/2], E4M3 scales [E, N, K/16] as bytes, float32 scale [E])."""
    E, N, K = w.shape
    g = w.float().view(E, N, K // 16, 16)
    amax = g.abs().amax(-1)
    scale2 = amax.amax((1, 2)) / (6.0 * 448.0)
    s = (amax / 6.0 / scale2.view(E, 1, 1)).clamp_(min=2.0 ** -9).to(torch.float8_e4m3fn)
    v = g / (s.float() * scale2.view(E, 1, 1)).unsqueeze(-1)
    code = torch.bucketize(v.abs(), torch.tensor(BORDERS, device=w.device)).to(torch.uint8)
    code |= (v < 0).to(torch.uint8) << 3
    code = code.view(E, N, K // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), s.view(torch.uint8).contiguous(), scale2.contiguous()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    T, E, k, K, N = (c[n] for n in ("T", "E", "k", "K", "N"))
    idx = _routing(c, gen)
    s = {"op": c["op"], "relu2": c["relu2"], "idx": idx}
    if c["op"] == "gemv":
        rows = (T, k, K) if c["per_slot"] else (T, K)
        s["x"] = torch.randn(*rows, device="cuda", dtype=dt, generator=gen)
        w = torch.randn(E, N, K, device="cuda", dtype=torch.bfloat16, generator=gen).mul_(K ** -0.5)
        s["w"], s["w_scale"], s["w_scale2"] = _quantise(w)
        s["y"] = torch.zeros(T, k, N, device="cuda", dtype=dt)
        return s
    count = torch.bincount(idx.flatten(), minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = count.cumsum(0)
    rows = T * k + c["tail"]
    s["off"], s["cap"], s["rows"] = off, int(count.max()), rows
    if c["op"] != "dgrad":
        s["x"] = _padded((rows,), K, dt, gen, 1.0)
    if c["op"] != "fwd":
        s["dy"] = _padded((rows,), N, dt, gen, 1.0)
    if c["op"] != "wgrad":
        s["w"] = _padded((E, N), K, dt, gen, K ** -0.5 if c["op"] == "fwd" else N ** -0.5)
    od = torch.float32 if c["out"] == "f32" else dt
    if c["op"] == "fwd":
        s["out"] = torch.zeros(rows, N, device="cuda", dtype=dt)
    elif c["op"] == "dgrad":
        s["out"] = torch.zeros(rows, K, device="cuda", dtype=dt)
    else:
        s["out"] = torch.zeros(E, N, K, device="cuda", dtype=od)
    return s


def _run_own(s):
    import mixture_experts_ffn_rmsnorm_b200 as moe
    if s["op"] == "fwd":
        moe.grouped_gemm(s["x"], s["w"], s["off"], s["out"], relu2=s["relu2"])
    elif s["op"] == "dgrad":
        moe.grouped_gemm_dgrad(s["dy"], s["w"], s["off"], s["out"])
    elif s["op"] == "wgrad":
        moe.grouped_gemm_wgrad(s["dy"], s["x"], s["off"], s["out"])
    else:
        moe.nvfp4_gemv(s["x"], s["idx"], s["w"], s["w_scale"], s["w_scale2"], s["y"], relu2=s["relu2"])
        return s["y"]
    return s["out"]


def _groups(s, t):
    """The rows of each expert, padded with zeros to the largest group: [E, cap, width] in 32 bits."""
    off = s["off"].long()
    at = off[:-1, None] + torch.arange(s["cap"], device=t.device)
    return torch.where((at < off[1:, None]).unsqueeze(-1), t.float()[at.clamp(max=s["rows"] - 1)], 0.0)


def _rows(s, g):
    """The inverse of _groups: [rows, width], zeros behind the last group."""
    off = s["off"].long()
    r = torch.arange(s["rows"], device=g.device)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True).clamp(max=off.numel() - 2)
    at = (r - off[e]).clamp(max=s["cap"] - 1)
    return torch.where((r < off[-1]).unsqueeze(-1), g[e, at], 0.0)


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "gemv":
        e = s["idx"].long().flatten()
        T, k = s["idx"].shape
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=e.device)
        packed = s["w"][e]
        w = torch.stack((table[(packed & 15).long()], table[(packed >> 4).long()]), -1)  # [T*k, N, K/2, 2]
        w = w.view(T * k, w.shape[1], -1, 16) * s["w_scale"][e].view(torch.float8_e4m3fn).float().unsqueeze(-1)
        x = s["x"].float()
        x = (x if x.dim() == 3 else x.unsqueeze(1).expand(T, k, -1)).reshape(T * k, -1, 1)
        y = torch.bmm(w.flatten(2), x).squeeze(-1) * s["w_scale2"][e].unsqueeze(-1)
        y = torch.relu(y).square() if s["relu2"] else y
        return y.view(T, k, -1).to(s["y"].dtype)
    if s["op"] == "fwd":
        y = torch.bmm(_groups(s, s["x"]), s["w"].float().transpose(1, 2))
        y = torch.relu(y).square() if s["relu2"] else y
        return _rows(s, y).to(s["out"].dtype)
    if s["op"] == "dgrad":
        return _rows(s, torch.bmm(_groups(s, s["dy"]), s["w"].float())).to(s["out"].dtype)
    return torch.bmm(_groups(s, s["dy"]).transpose(1, 2), _groups(s, s["x"])).to(s["out"].dtype)


def work(case):
    c = case
    T, E, k, K, N = (c[n] for n in ("T", "E", "k", "K", "N"))
    rows = T * k
    touched = E * (1.0 - (1.0 - k / E) ** T)  # expected number of experts with a row
    flops = 2.0 * rows * K * N
    if c["op"] == "gemv":
        x = (rows if c["per_slot"] else T) * K * 2
        return {"bytes": touched * (N * K * 9 / 16 + 4) + x + rows * (N * 2 + 4), "flops": flops}
    if c["op"] == "wgrad":
        return {"bytes": rows * (K + N) * 2 + E * N * K * (4 if c["out"] == "f32" else 2) + (E + 1) * 4, "flops": flops}
    return {"bytes": rows * (K + N) * 2 + touched * N * K * 2 + (E + 1) * 4, "flops": flops}


def exact(case, seed):
    """The definition in 64 bits, one expert after the other."""
    s = prepare(case, seed)
    if case["op"] == "gemv":
        T, k = s["idx"].shape
        y = torch.zeros(T, k, case["N"], device="cuda", dtype=torch.float64)
        for e in torch.unique(s["idx"]).tolist():
            byte = s["w"][e].to(torch.int32)
            code = torch.empty(case["N"], case["K"], dtype=torch.int32, device="cuda")
            code[:, 0::2] = byte % 16
            code[:, 1::2] = byte // 16
            ex, man = (code // 2) % 4, (code % 2).double()
            mag = torch.where(ex == 0, man / 2, (1 + man / 2) * torch.exp2(ex.double() - 1))
            w = torch.where(code >= 8, -mag, mag)
            scale = s["w_scale"][e].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
            w = w * scale * s["w_scale2"][e].double()
            for t, j in (s["idx"] == e).nonzero().tolist():
                x = s["x"][t, j] if case["per_slot"] else s["x"][t]
                y[t, j] = w @ x.double()
        return y.clamp(min=0) ** 2 if case["relu2"] else y
    off = s["off"].tolist()
    r = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if case["op"] == "wgrad":
            r[e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
        elif case["op"] == "dgrad":
            r[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
        else:
            r[a:b] = s["x"][a:b].double() @ s["w"][e].double().T
    return r.clamp(min=0) ** 2 if case["op"] == "fwd" and case["relu2"] else r
