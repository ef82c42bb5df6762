"""CPU-side checks of the C ABI: the library builds and loads without a GPU,
exports every function include/*.h declares, and its host-side validation
answers before touching a device."""
import ctypes
import glob
import os
import re

import pytest

import mixture_experts_ffn_rmsnorm_b200 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def declared_functions():
    names = []
    for h in glob.glob(os.path.join(ROOT, "include", "*.h")):
        src = open(h).read()
        names += re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", src)
    return sorted(set(names))


def test_header_declares_the_boundary():
    names = declared_functions()
    for required in ("moe_create", "moe_forward", "moe_destroy"):
        assert required in names
    assert set(names) == set(moe.EXPORTED_SYMBOLS)


def test_library_exports_every_declared_symbol():
    lib = moe.load_library()
    for name in declared_functions():
        assert hasattr(lib, name), name


def test_status_strings():
    lib = moe.load_library()
    for code in range(9):
        s = lib.moe_status_string(code)
        assert s and s != b"unknown status"
    assert lib.moe_status_string(99) == b"unknown status"


def _cfg(**kw):
    base = dict(hidden_size=256, num_experts=8, top_k=2, moe_inter=128, shared_inter=256,
                latent_size=0, max_tokens=16, rms_eps=1e-5, routed_scaling_factor=1.0,
                expert_wdtype=0)
    base.update(kw)
    return moe.MoEConfig(**base)


def _create(cfg, w):
    lib = moe.load_library()
    h = ctypes.c_void_p(1234)
    st = lib.moe_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h))
    return st, h


ALL16 = dict(norm_w=16, gate_w=32, gate_bias=None, up_w=48, down_w=64, up_scale=None,
             down_scale=None, shared_up_w=80, shared_down_w=96, fc1_w=None, fc2_w=None)


@pytest.mark.parametrize("bad", [dict(top_k=0), dict(top_k=9), dict(top_k=17, num_experts=32),
                                 dict(num_experts=257, top_k=2), dict(hidden_size=100),
                                 dict(moe_inter=96), dict(shared_inter=0), dict(latent_size=-64),
                                 dict(latent_size=32), dict(max_tokens=0), dict(rms_eps=-1.0),
                                 dict(expert_wdtype=5), dict(shared_wdtype=3),
                                 dict(latent_wdtype=-1),
                                 dict(routed_scaling_factor=float("inf"))])
def test_invalid_configs_rejected_on_host(bad):
    # NemotronMoeLayer `new`: top_k must be in 1..=num_experts and within the
    # routing kernels' bounds; plus this library's layout requirements.
    st, h = _create(_cfg(**bad), moe.MoEWeights(**ALL16))
    assert st == 1 and h.value is None


def test_null_and_misaligned_weights_rejected():
    w = dict(ALL16)
    w["up_w"] = None
    st, h = _create(_cfg(), moe.MoEWeights(**w))
    assert st == 2 and h.value is None
    w = dict(ALL16)
    w["gate_w"] = 34
    st, _ = _create(_cfg(), moe.MoEWeights(**w))
    assert st == 3
    # FP8 needs the row scales; LatentMoE needs fc1/fc2
    st, _ = _create(_cfg(expert_wdtype=1), moe.MoEWeights(**ALL16))
    assert st == 2
    st, _ = _create(_cfg(latent_size=128), moe.MoEWeights(**ALL16))
    assert st == 2
    # FP8 shared expert / fc1 / fc2 need their row scales too
    st, _ = _create(_cfg(shared_wdtype=1), moe.MoEWeights(**ALL16))
    assert st == 2
    lat = dict(ALL16, fc1_w=112, fc2_w=128)
    st, _ = _create(_cfg(latent_size=128, latent_wdtype=1), moe.MoEWeights(**lat))
    assert st == 2
    # FP8 routed experts are wired for the direct layer only
    st, _ = _create(_cfg(latent_size=128, expert_wdtype=1),
                    moe.MoEWeights(**dict(lat, up_scale=144, down_scale=160)))
    assert st == 1


def test_invalid_handle_rejected():
    lib = moe.load_library()
    assert lib.moe_forward(None, None, None, 1, None) == 8
    assert lib.moe_destroy(None) == 8
    bogus = ctypes.create_string_buffer(64)
    assert lib.moe_forward(ctypes.addressof(bogus), None, None, 1, None) == 8
    assert lib.moe_last_launch_count(None) == -1


def test_static_sort_validates_on_host():
    # every rejection happens before the device is touched
    lib = moe.load_library()
    p = 256  # any non-NULL value: nothing is dereferenced on these paths
    assert lib.moe_sort_static(None, 10, 2, 8, p, p, p, None, None) == 2
    assert lib.moe_sort_static(p, 10, 2, 8, p, None, p, None, None) == 2
    assert lib.moe_sort_static(p, 8193, 2, 8, p, p, p, None, None) == 4
    assert lib.moe_sort_static(p, 0, 2, 8, p, p, p, None, None) == 4
    assert lib.moe_sort_static(p, 10, 0, 8, p, p, p, None, None) == 1
    assert lib.moe_sort_static(p, 10, 17, 64, p, p, p, None, None) == 1
    assert lib.moe_sort_static(p, 10, 4, 257, p, p, p, None, None) == 1
    assert lib.moe_sort_static(p, 10, 9, 8, p, p, p, None, None) == 1


def test_missing_library_fails_loudly():
    # no fallback: a library path that does not exist is an error, in a fresh
    # interpreter (the loaded library is cached per process)
    import subprocess
    import sys
    code = ("import mixture_experts_ffn_rmsnorm_b200 as m\n"
            "try:\n"
            "    m.load_library()\n"
            "except FileNotFoundError as e:\n"
            "    print('raised', e)\n"
            "else:\n"
            "    print('loaded')\n")
    env = dict(os.environ, MOE_B200_LIBRARY="/nonexistent/libmoe_b200.so")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("raised"), r.stdout


def test_grouped_gemm_validates_on_host():
    # every rejection happens before the device is touched; 256 stands for any pointer
    lib = moe.load_library()
    p = 256

    def fwd(x=p, ldx=64, w=p, ldw=64, off=p, E=4, rows=8, K=64, N=48, dt=0, act=0, y=p, ldy=48):
        return lib.moe_grouped_gemm(x, ldx, w, ldw, off, E, rows, K, N, dt, act, y, ldy, None, None)

    def dgrad(dy=p, lddy=48, w=p, ldw=64, off=p, E=4, rows=8, K=64, N=48, dt=0, dx=p, lddx=64):
        return lib.moe_grouped_gemm_dgrad(dy, lddy, w, ldw, off, E, rows, K, N, dt, dx, lddx, None,
                                          None)

    def wgrad(dy=p, lddy=48, x=p, ldx=64, off=p, E=4, rows=8, K=64, N=48, dt=0, dw=p, lddw=64,
              odt=0, acc=0):
        return lib.moe_grouped_gemm_wgrad(dy, lddy, x, ldx, off, E, rows, K, N, dt, dw, lddw, odt,
                                          acc, None, None)

    for f, ptrs, lds in ((fwd, ("x", "w", "off", "y"), ("ldx", "ldw", "ldy")),
                         (dgrad, ("dy", "w", "off", "dx"), ("lddy", "ldw", "lddx")),
                         (wgrad, ("dy", "x", "off", "dw"), ("lddy", "ldx", "lddw"))):
        for name in ptrs:
            assert f(**{name: None}) == 2, name
            assert f(**{name: 257}) == 3, name
        for name in lds:
            assert f(**{name: 40}) == 1, name           # narrower than the row
            assert f(**{name: 1 << 22}) == 1, name
        for name in lds[:2]:
            assert f(**{name: 68}) == 1, name           # an operand's stride off 16 bytes
        for bad in (dict(E=0), dict(E=257), dict(K=0), dict(N=0), dict(K=-1), dict(N=131073),
                    dict(dt=2), dict(dt=-1)):
            assert f(**bad) == 1, bad
        assert f(rows=-1) == 4
        assert f(rows=16777217) == 4
    assert fwd(act=2) == 1
    assert wgrad(odt=1) == 1          # neither the operands' type nor float32
    assert wgrad(acc=1) == 1          # accumulation wants float32
    assert wgrad(odt=2, acc=2) == 1
    assert wgrad(odt=2, dw=258) == 3  # float32 elements
    assert fwd(rows=0, x=None, y=None) == 0   # nothing to do
    assert dgrad(rows=0, dy=None, dx=None) == 0


def test_nvfp4_gemv_validates_on_host():
    lib = moe.load_library()
    p = 256

    def gemv(x=p, ldx=64, per_slot=0, idx=p, T=2, k=3, w=p, ws=p, ws2=p, E=4, K=64, N=24, dt=0,
             act=0, y=p, ldy=24):
        return lib.moe_nvfp4_gemv(x, ldx, per_slot, idx, T, k, w, ws, ws2, E, K, N, dt, act, y, ldy,
                                  None, None)

    for name in ("x", "idx", "w", "ws", "ws2", "y"):
        assert gemv(**{name: None}) == 2, name
        assert gemv(**{name: 257}) == 3, name
    for bad in (dict(E=0), dict(E=257), dict(k=0), dict(k=17), dict(K=0), dict(K=48), dict(K=8224),
                dict(N=0), dict(N=131073), dict(dt=2), dict(act=2), dict(per_slot=2), dict(ldx=56),
                dict(ldx=66), dict(ldy=23)):
        assert gemv(**bad) == 1, bad
    assert gemv(T=-1) == 4
    assert gemv(T=342) == 4  # 1026 routed rows
    assert gemv(T=0, x=None, y=None) == 0


def refused(code, f, *a, **kw):
    with pytest.raises(moe.MoEError) as ei:
        f(*a, **kw)
    assert ei.value.status == code


def test_grouped_gemm_wrappers_refuse_bad_tensors():
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32)
    x, w, y, dw = z(8, 64), z(2, 48, 64), z(8, 48), z(2, 48, 64)
    for f, a in ((moe.grouped_gemm, (x, w, off, y)), (moe.grouped_gemm_dgrad, (y, w, off, x)),
                 (moe.grouped_gemm_wgrad, (y, x, off, dw))):
        refused(7, f, *a)  # good shapes, but not on the device
        for i in range(4):
            flat = list(a)
            flat[i] = flat[i].reshape(-1)[:-1]
            refused(1, f, *flat)
        refused(1, f, a[0].double(), *a[1:])
        refused(1, f, a[0], a[1].half(), *a[2:])
        refused(1, f, *a[:2], off.long(), a[3])
        refused(1, f, *a[:3], a[3].double())
        refused(1, f, *a, status=z(1))
        refused(1, f, a[0][:7], *a[1:])
    refused(1, moe.grouped_gemm, x, z(1, 48, 64).expand(2, 48, 64), off, y)  # one matrix for all
    refused(1, moe.grouped_gemm, x, w.transpose(1, 2), off, z(8, 64))
    refused(1, moe.grouped_gemm, z(64, 8).T, w, off, y)


def test_nvfp4_gemv_wrapper_refuses_bad_tensors():
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    good = [z(2, 64), z(2, 3, dt=torch.int32), z(4, 24, 32, dt=torch.uint8),
            z(4, 24, 4, dt=torch.uint8), z(4, dt=torch.float32), z(2, 3, 24)]
    refused(7, moe.nvfp4_gemv, *good)  # good shapes, but not on the device
    bad = [(0, z(2, 32)), (0, z(2, 1, 64)), (0, z(64)), (0, z(2, 64, dt=torch.float64)),
           (1, z(2, 3, dt=torch.int64)), (1, z(6, dt=torch.int32)),
           (2, z(4, 24, 32, dt=torch.int8)), (2, z(24, 32, dt=torch.uint8)),
           (2, z(4, 24, 64, dt=torch.uint8)[..., :32]), (3, z(4, 24, 3, dt=torch.uint8)),
           (3, z(4, 24, 4)), (4, z(3, dt=torch.float32)), (4, z(4)), (5, z(2, 3, 25)),
           (5, z(2, 3, 24, dt=torch.float16)), (5, z(6, 24))]
    for i, t in bad:
        refused(1, moe.nvfp4_gemv, *good[:i], t, *good[i + 1:])
    refused(1, moe.nvfp4_gemv, *good, status=z(1))
