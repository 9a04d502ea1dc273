"""Checks of the C entry points of the attention layer in 8 bits that need no GPU:
argument validation returns the documented status before anything is enqueued, the
rotation's table against extended precision, and the oracle's own closed forms."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from nvfp4_w4a4_gemm_quantize_amd import binding
from oracle import layer8 as O8

OK, EINVAL, ESHAPE, EALIGN, EUNSUPPORTED, EHIP, ESIZE = 0, -1, -2, -3, -4, -5, -6
A16, B16, MIS = 0x10000, 0x900000, 0x10002
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("validation tests with fake device pointers run on GPU-less hosts only")
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libnvfp4.so is not built; run __graft_entry__.build() first")
    return binding.load()


def steps(lib, dim=64, base=10000.0, scaling=0, factor=1.0, original=8192.0, slow=1.0, fast=4.0, factors=None, no_steps=False):
    s, amp = (ctypes.c_uint64 * 512)(), ctypes.c_double()
    f = None if factors is None else (ctypes.c_double * len(factors))(*factors)
    rc = lib.rotary_steps(dim, base, scaling, factor, original, slow, fast, f, None if no_steps else s, ctypes.byref(amp))
    return rc, [int(x) for x in s[:max(dim, 0) // 2]], amp.value


def test_rotary_steps_validation(lib):
    assert steps(lib)[0] == OK
    for bad in (dict(dim=0), dict(dim=-16)):
        assert steps(lib, **bad)[0] == ESHAPE, bad
    for bad in (dict(dim=8), dict(dim=24), dict(dim=1040)):
        assert steps(lib, **bad)[0] == EUNSUPPORTED, bad
    for bad in (dict(base=1.0), dict(base=NAN), dict(base=INF), dict(scaling=-1), dict(scaling=5), dict(scaling=1, factor=0.5),
                dict(scaling=2, factor=NAN), dict(scaling=3, factor=INF), dict(scaling=3, factor=2.0, original=0.0),
                dict(scaling=4, factor=2.0, slow=0.0), dict(scaling=4, factor=2.0, slow=4.0), dict(scaling=3, factor=2.0, fast=INF),
                dict(scaling=3, factor=2.0, original=NAN), dict(factors=[1.0] * 31 + [0.0]), dict(factors=[1.0] * 31 + [INF]),
                dict(factors=[NAN] * 32), dict(no_steps=True)):
        assert steps(lib, **bad)[0] == EINVAL, bad
    assert steps(lib, factor=NAN)[0] == OK      # not read without a scaling


@pytest.mark.parametrize("dim", [16, 32, 64, 96, 128, 1024])
@pytest.mark.parametrize("kw", [dict(), dict(base=1e6), dict(base=1.5), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0), dict(scaling="yarn", factor=1.0), dict(scaling="wavelength", factor=8.0),
                                dict(scaling="yarn", factor=4.0, original=256.0, slow=0.5, fast=60.0), dict(pair_factors=1.25)])
def test_rotary_steps_are_the_formulas(lib, dim, kw):
    kw = dict(kw)
    if "pair_factors" in kw:
        kw["pair_factors"] = [kw["pair_factors"] ** i % 7 + 0.25 for i in range(dim // 2)]
    names = ["none", "linear", "ntk", "yarn", "wavelength"]
    turn, amp = O8.turns(dim, **kw)
    args = {"scaling": names.index(kw.get("scaling", "none")), "base": kw.get("base", 10000.0), "factor": kw.get("factor", 1.0),
            "original": kw.get("original", 8192.0), "slow": kw.get("slow", 1.0), "factors": kw.get("pair_factors"),
            "fast": kw.get("fast", 32.0 if kw.get("scaling") == "yarn" else 4.0)}
    rc, got, amplitude = steps(lib, dim, **args)
    assert rc == OK and abs(amplitude - amp) < 1e-14
    frac = np.array(got, dtype=np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64
    # both in extended precision: a few of its units apart, whole turns aside
    off = np.abs(frac - np.mod(turn, 1))
    assert (np.minimum(off, 1 - off) < 2.0 ** -60).all()


def test_rotary_steps_known_values(lib):
    """Pair 0 turns by one radian; a factor of 2 pi makes that 1 / 2 pi squared of a turn; whole turns vanish."""
    one = steps(lib, 16)[1][0]
    assert abs(one / 2.0 ** 64 - 1 / (2 * np.pi)) < 1e-15
    assert steps(lib, 16, scaling=1, factor=2.0)[1][0] in range(one // 2 - 1, one // 2 + 2)
    assert steps(lib, 16, factors=[0.5 / (2 * np.pi)] * 8)[1][0] < 2 ** 14 or steps(lib, 16, factors=[0.5 / (2 * np.pi)] * 8)[1][0] > 2 ** 64 - 2 ** 14


def rot(lib, x=A16, ld=256, T=4, heads=2, dim=128, pos=A16, st=A16, rd=128, layout=0, amp=1.0, out=B16, ldo=256):
    return lib.rotary(x, ld, T, heads, dim, pos, st, rd, layout, amp, out, ldo, None)


def test_rotary_validation(lib):
    for bad in (dict(T=-1), dict(heads=0), dict(dim=0), dict(ld=255), dict(ldo=248), dict(rd=144), dict(rd=0), dict(rd=-2)):
        assert rot(lib, **bad) == ESHAPE, bad
    for bad in (dict(dim=120, rd=16), dict(dim=1040, ld=4096, ldo=4096), dict(rd=24), dict(heads=65537), dict(T=2 ** 31)):
        assert rot(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(x=None), dict(out=None), dict(pos=None), dict(st=None), dict(layout=2), dict(amp=NAN), dict(amp=INF),
                dict(out=A16, ldo=264)):
        assert rot(lib, **bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(out=0x10008), dict(ld=260), dict(ldo=260), dict(pos=MIS), dict(st=0x10004)):
        assert rot(lib, **bad) == EALIGN, bad
    assert rot(lib, T=0, x=None, out=None, pos=None, st=None) == OK
    assert rot(lib, out=A16) == EHIP            # in place: valid, but no GPU here


def append(lib, q=None, ldq=512, hq=0, qo=None, ldqo=512, k=A16, ldk=256, v=A16, ldv=256, pos=A16, slots=A16, T=4, st=A16, rd=64,
           layout=1, amp=1.0, kc=A16, vc=A16, dt=2, pages=4, page=16, heads=2, dim=128, ps=4096, hs=2048, ts=128, ks=None, vs=None,
           kb=A16, vb=A16):
    return lib.paged_kv_append(q, ldq, hq, qo, ldqo, k, ldk, v, ldv, pos, slots, T, st, rd, layout, amp, kc, vc, dt, pages, page, heads,
                               dim, ps, hs, ts, ks, vs, kb, vb, None)


def test_append_validation(lib):
    for dt in (2, 3):
        assert append(lib, dt=dt) == EHIP       # valid
        for bad in (dict(kb=None), dict(vb=None), dict(ks=A16), dict(vs=A16)):
            assert append(lib, dt=dt, **bad) == EINVAL, bad
    for dt in (0, 1):
        assert append(lib, dt=dt, kb=None, vb=None) == EHIP
        assert append(lib, dt=dt) == EINVAL
    assert append(lib, dt=1, kb=None, vb=None, ks=A16, vs=A16) == EHIP
    for bad in (dict(T=-1), dict(heads=0), dict(pages=0), dict(dim=0), dict(ldk=255), dict(ldv=0), dict(ts=127), dict(hq=-1),
                dict(hq=4, q=A16, qo=B16, ldq=511), dict(rd=144), dict(rd=-16)):
        assert append(lib, **bad) == ESHAPE, bad
    for bad in (dict(dim=96, ts=96, hs=96 * 16), dict(page=20), dict(page=8), dict(T=2 ** 31), dict(rd=40)):
        assert append(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(dt=4), dict(dt=-1), dict(pos=None),
                dict(st=None), dict(layout=-1), dict(amp=NAN), dict(hq=4, q=A16), dict(hq=4, qo=B16), dict(q=A16), dict(rd=0),
                dict(hq=4, q=A16, qo=A16, ldqo=520)):
        assert append(lib, **bad) == EINVAL, bad
    for bad in (dict(k=MIS), dict(ldk=260), dict(kc=0x10008), dict(ts=136), dict(slots=0x10004), dict(hq=4, q=MIS, qo=B16), dict(pos=MIS)):
        assert append(lib, **bad) == EALIGN, bad
    assert append(lib, rd=0, st=None, pos=None) == EHIP
    assert append(lib, T=0, k=None, v=None, slots=None, pos=None, st=None) == OK


def attn(lib, q=A16, ldq=512, T=4, qs=A16, sl=A16, R=2, mn=2, ms=100, hq=4, kc=A16, vc=A16, dt=2, pages=4, page=16, heads=2,
         dim=128, ps=4096, hs=2048, ts=128, kb=A16, vb=A16, table=A16, MP=8, ld=8, scale=0.1, window=0, out=A16, od=1, ldo=512,
         lse=None, ws=A16, nws=None):
    if nws is None:
        nws = lib.paged_attention_workspace_bytes(T, R, hq, heads, dim, mn, ms)
    return lib.paged_attention_blocks(q, ldq, T, qs, sl, R, mn, ms, hq, kc, vc, dt, pages, page, heads, dim, ps, hs, ts, kb, vb, table,
                                      MP, ld, scale, window, out, od, ldo, lse, ws, nws, None)


def test_attention_validation(lib):
    for dt in (2, 3):
        assert attn(lib, dt=dt) == EHIP
    for bad in (dict(T=-1), dict(R=-1), dict(hq=3), dict(heads=0), dict(mn=-1), dict(ldq=511), dict(MP=0, ld=0), dict(pages=0)):
        assert attn(lib, **bad) == ESHAPE, bad
    for bad in (dict(dim=80), dict(page=17), dict(T=2 ** 30)):
        assert attn(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(q=None), dict(qs=None), dict(sl=None), dict(kc=None), dict(vc=None), dict(kb=None), dict(vb=None), dict(table=None),
                dict(out=None), dict(ws=None), dict(od=5), dict(dt=0), dict(dt=1), dict(dt=4), dict(window=-1), dict(scale=INF)):
        assert attn(lib, **bad) == EINVAL, bad
    for bad in (dict(q=MIS), dict(ldq=516), dict(out=0x10008), dict(ldo=514), dict(lse=MIS), dict(ws=0x10008), dict(table=MIS), dict(ts=136)):
        assert attn(lib, **bad) == EALIGN, bad
    assert attn(lib, nws=100) == ESIZE
    assert attn(lib, T=0, q=None, out=None) == OK and attn(lib, R=0, qs=None) == OK


def quant(lib, x=A16, rows=4, cols=256, ld=256, c=A16, s=A16):
    return lib.int8_quantize(x, rows, cols, ld, c, s, None)


def gemm(lib, a=A16, sa=A16, m=4, w=A16, sw=A16, n=24, k=256, out=A16, od=1, ldo=24, ws=None, nws=0):
    return lib.gemm_w8a8(a, sa, m, w, sw, n, k, out, od, ldo, ws, nws, None)


def linear(lib, x=A16, m=4, k=256, ld=256, a=A16, sa=A16, w=A16, sw=A16, n=24, out=A16, od=1, ldo=24, ws=None, nws=0):
    return lib.int8_linear(x, m, k, ld, a, sa, w, sw, n, out, od, ldo, ws, nws, None)


def test_int8_validation(lib):
    assert quant(lib) == EHIP and gemm(lib) == EHIP and linear(lib) == EHIP
    for bad in (dict(rows=-1), dict(cols=0), dict(ld=255)):
        assert quant(lib, **bad) == ESHAPE, bad
    for bad in (dict(cols=250), dict(cols=131072, ld=131072), dict(rows=2 ** 31)):
        assert quant(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(x=None), dict(c=None), dict(s=None)):
        assert quant(lib, **bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(ld=260), dict(c=0x10008), dict(s=MIS)):
        assert quant(lib, **bad) == EALIGN, bad
    for bad in (dict(m=-1), dict(n=0), dict(k=0), dict(ldo=23)):
        assert gemm(lib, **bad) == ESHAPE, bad
        assert linear(lib, **bad) == ESHAPE, bad
    for bad in (dict(k=264), dict(k=1 << 17, **{}), dict(m=2 ** 31), dict(n=2 ** 31, ldo=2 ** 31), dict(m=2 ** 31 - 1, n=2 ** 20, ldo=2 ** 20)):
        assert gemm(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None), dict(od=2)):
        assert gemm(lib, **bad) == EINVAL, bad
        assert linear(lib, **bad) == EINVAL, bad
    for bad in (dict(a=0x10008), dict(w=MIS), dict(sa=MIS), dict(sw=MIS), dict(out=0x10001), dict(od=0, out=MIS)):
        assert gemm(lib, **bad) == EALIGN, bad
        assert linear(lib, **bad) == EALIGN, bad
    assert linear(lib, x=None) == EINVAL and linear(lib, x=MIS) == EALIGN and linear(lib, ld=248) == ESHAPE
    big = dict(m=40, n=512, k=4096)
    need = lib.gemm_w8a8_workspace_bytes(40, 512, 4096)
    assert need > 0 and lib.gemm_w8a8_workspace_bytes(-1, 512, 4096) == 0 and lib.gemm_w8a8_workspace_bytes(40, 512, 4095) == 0
    for f in (gemm, linear):
        more = dict(ldo=512, **(dict(ld=4096) if f is linear else {}), **big)
        assert f(lib, ws=A16, nws=need, **more) == EHIP and f(lib, **more) == EHIP
        assert f(lib, ws=A16, nws=need - 1, **more) == ESIZE and f(lib, ws=0x10008, nws=need, **more) == EALIGN
    assert quant(lib, rows=0, x=None, c=None, s=None) == OK
    assert gemm(lib, m=0, a=None, sa=None, out=None) == OK and linear(lib, m=0, x=None, a=None, sa=None, out=None) == OK


def test_layer8_abi_layer_under_address_and_ub_sanitizers(tmp_path):
    """abi_layer8.cpp and its validation built for the host alone with ASan and UBSan, launchers stubbed."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "nvfp4_w4a4_gemm_quantize_amd", "csrc")
    exe = str(tmp_path / "layer8_host_check")
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           os.path.join(root, "tests", "layer8_host_check.cpp"), os.path.join(csrc, "abi_layer8.cpp"),
           os.path.join(csrc, "validate_layer8.cpp"), os.path.join(csrc, "validate_serving.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "cases ok" in r.stdout, r.stdout + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-4000:]


def test_binding_refuses_cpu_tensors():
    import torch
    x, i = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    cache, scale = torch.zeros((2, 1, 16, 128), dtype=torch.int8), torch.zeros((2, 1, 1), dtype=torch.uint8).view(torch.float8_e8m0fnu)
    table = binding.RotaryTable(torch.zeros(64, dtype=torch.int64), 128, "half", 1.0)
    for call in (lambda: binding.rotary(x, i, table, 128),
                 lambda: binding.paged_kv_append(x, x, i, i.long(), cache, cache, rotation=table, k_scale=scale, v_scale=scale),
                 lambda: binding.paged_attention_blocks(x, cache, cache, scale, scale, i.view(2, 2), i[:3], i[:2], 2, 8),
                 lambda: binding.int8_quantize(x), lambda: binding.int8_linear(x, cache[0, 0], x[0].float()),
                 lambda: binding.gemm_w8a8(cache[0, 0], x[0].float(), cache[0, 0], x[0].float())):
        with pytest.raises(binding.NVFP4Error):
            call()


def test_rotary_table_refuses(lib):
    for bad in (dict(layout="other"), dict(scaling="other"), dict(rotary_dim=20), dict(pair_factors=[1.0]), dict(factor=0.5, scaling="ntk")):
        with pytest.raises(binding.NVFP4Error):
            binding.rotary_table(**{**dict(rotary_dim=64, device="cpu"), **bad})
    t = binding.rotary_table(64, device="cpu", layout="interleaved", scaling="yarn", factor=2.0, amplitude=3.0)
    assert t.steps.shape == (32,) and t.amplitude == 3.0 and t.layout == "interleaved" and t.rotary_dim == 64


# ------------------------------------------------------------ oracle pins --

def test_oracle_rotation_closed_forms():
    """Lengths of pairs stay, scores depend on the distance of positions alone, a quarter turn swaps."""
    rng = np.random.default_rng(0)
    turn, _ = O8.turns(32)
    q, k = rng.standard_normal((1, 1, 40)), rng.standard_normal((1, 1, 40))
    for layout in ("half", "interleaved"):
        dots = [float((O8.rotate(q, [a], turn, layout)[0] * O8.rotate(k, [b], turn, layout)[0]).sum()) for a, b in ((9, 4), (105, 100), (5, 0))]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-12)
        y, _ = O8.rotate(np.eye(40)[None], [1], np.full(16, 0.25), layout)
        assert abs(y[0, 0, 16 if layout == "half" else 1] - 1) < 1e-15 and abs(y[0, 35, 35] - 1) < 1e-15


def test_oracle_codes_worked_examples():
    assert O8.round_codes(np.array([1.0625, 1.1875, 17.0, 19.0, 449.0, -1000.0, 2.0 ** -10, 2.0 ** -10 * 1.01]), "e4m3").tolist() == \
        [1.0, 1.25, 16.0, 20.0, 448.0, -448.0, 0.0, 2.0 ** -9]
    assert O8.round_codes(np.array([0.5, 1.5, -2.5, 127.5, 300.0, np.nan]), "int8").tolist() == [0.0, 2.0, -2.0, 127.0, 127.0, 0.0]
    assert [O8.scale_byte(x, "int8") for x in (0.0, 127.0, 127.0001, 63.5, 2.0 ** -140)] == [1, 127, 128, 126, 1]
    assert [O8.scale_byte(x, "e4m3") for x in (448.0, 448.1, 1.75)] == [127, 128, 119]


def test_oracle_append_worked_example():
    """A token of 100, then one of 300 beside it: the first one's code halves; a new first token begins the block."""
    codes, scales = np.full((1, 1, 16, 2), 5.0), np.full((1, 1, 1), 130, np.uint8)
    c, s = O8.append(np.array([[[100.0, -50.0]]]), [0], codes, scales, "int8")
    assert s[0, 0, 0] == 127 and c[0, 0, 0].tolist() == [100, -50] and (c[0, 0, 1:] == 0).all()
    c, s = O8.append(np.array([[[300.0, 1.0]]]), [1], c, s, "int8")
    assert s[0, 0, 0] == 129 and c[0, 0, :2].tolist() == [[25, -12], [75, 0]]
    np.testing.assert_allclose(O8.block_values(c, s)[0, 0, :2], [[100, -48], [300, 0]])


def test_oracle_int8_worked_example():
    c, s = O8.int8_quantize([[127.0, 63.5, -0.5, 1.5]])
    assert c.tolist() == [[127, 64, 0, 2]] and s[0] == 1.0
    assert O8.gemm_w8a8(c, s, c, np.array([0.5], np.float32)).tolist() == [[(127 ** 2 + 64 ** 2 + 4) / 2]]
