"""Checks of the paged serving step's C entry points that need no GPU: argument
validation returns the documented status before anything is enqueued, workspace
sizes, and the oracle's own small closed forms."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from nvfp4_w4a4_gemm_quantize_amd import binding
from oracle import paged as OP

OK, EINVAL, ESHAPE, EALIGN, EUNSUPPORTED, EHIP, ESIZE = 0, -1, -2, -3, -4, -5, -6
A16, MIS = 0x10000, 0x10002


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("validation tests with fake device pointers run on GPU-less hosts only")
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libnvfp4.so is not built; run __graft_entry__.build() first")
    return binding.load()


def plan(lib, ctx=A16, new=A16, R=4, page=16, free=A16, F=10, cur=None, table=A16, MP=8, ld=8, qs=A16, sl=A16, pos=A16,
         slots=A16, T=16, counts=A16):
    return lib.paged_plan(ctx, new, R, page, free, F, cur, table, MP, ld, qs, sl, pos, slots, T, counts, None)


def test_plan_validation(lib):
    for bad in (dict(R=-1), dict(F=-1), dict(MP=-1), dict(T=-1), dict(ld=7), dict(page=0)):
        assert plan(lib, **bad) == ESHAPE, bad
    for bad in (dict(page=8), dict(page=24), dict(page=2048), dict(T=2 ** 31), dict(R=2 ** 31), dict(MP=2 ** 31, ld=2 ** 31)):
        assert plan(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(ctx=None), dict(new=None), dict(free=None), dict(table=None), dict(qs=None), dict(sl=None), dict(pos=None),
                dict(slots=None), dict(counts=None)):
        assert plan(lib, **bad) == EINVAL, bad
    for bad in (dict(ctx=MIS), dict(slots=0x10004), dict(table=MIS), dict(cur=MIS)):
        assert plan(lib, **bad) == EALIGN, bad


def write(lib, k=A16, ldk=256, v=A16, ldv=256, slots=A16, T=4, kc=A16, vc=A16, dt=0, pages=4, page=16, heads=2, dim=128,
          ps=4096, hs=2048, ts=128, ks=None, vs=None):
    return lib.paged_kv_write(k, ldk, v, ldv, slots, T, kc, vc, dt, pages, page, heads, dim, ps, hs, ts, ks, vs, None)


def test_kv_write_validation(lib):
    for bad in (dict(T=-1), dict(heads=0), dict(pages=0), dict(dim=0), dict(ldk=255), dict(ldv=0), dict(ts=127), dict(ps=-8)):
        assert write(lib, **bad) == ESHAPE, bad
    for bad in (dict(dim=96, ts=96, hs=96 * 16), dict(page=20), dict(T=2 ** 31), dict(ts=2 ** 27), dict(ps=2 ** 36)):
        assert write(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(dt=2), dict(ks=A16)):
        assert write(lib, **bad) == EINVAL, bad
    for bad in (dict(k=MIS), dict(ldk=260), dict(kc=0x10008), dict(ts=132), dict(hs=2052), dict(slots=0x10004),
                dict(dt=1, ts=136), dict(dt=1, ks=MIS)):
        assert write(lib, **bad) == EALIGN, bad
    assert write(lib, T=0, k=None, v=None, slots=None) == OK


def attn(lib, q=A16, ldq=512, T=4, qs=A16, sl=A16, R=2, mn=2, ms=100, hq=4, kc=A16, vc=A16, dt=0, pages=4, page=16, heads=2,
         dim=128, ps=4096, hs=2048, ts=128, table=A16, MP=8, ld=8, scale=0.1, window=0, ks=None, vs=None, out=A16, od=1,
         ldo=512, lse=None, ws=A16, nws=None):
    if nws is None:
        nws = lib.paged_attention_workspace_bytes(T, R, hq, heads, dim, mn, ms)
    return lib.paged_attention(q, ldq, T, qs, sl, R, mn, ms, hq, kc, vc, dt, pages, page, heads, dim, ps, hs, ts, table, MP,
                               ld, scale, window, ks, vs, out, od, ldo, lse, ws, nws, None)


def test_attention_validation(lib):
    for bad in (dict(T=-1), dict(R=-1), dict(hq=3), dict(hq=0), dict(heads=0), dict(mn=-1), dict(ms=-1), dict(ldq=511),
                dict(ldo=508), dict(MP=0, ld=0), dict(ld=7), dict(pages=0)):
        assert attn(lib, **bad) == ESHAPE, bad
    for bad in (dict(dim=80), dict(page=17), dict(T=2 ** 30), dict(MP=2 ** 31, ld=2 ** 31)):
        assert attn(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(q=None), dict(qs=None), dict(sl=None), dict(kc=None), dict(vc=None), dict(table=None), dict(out=None),
                dict(ws=None), dict(od=5), dict(dt=3), dict(window=-1), dict(scale=float("inf")), dict(ks=A16)):
        assert attn(lib, **bad) == EINVAL, bad
    for bad in (dict(q=MIS), dict(ldq=516), dict(out=0x10008), dict(ldo=514), dict(lse=MIS), dict(ws=0x10008), dict(table=MIS)):
        assert attn(lib, **bad) == EALIGN, bad
    assert attn(lib, nws=100) == ESIZE
    assert attn(lib, T=0, q=None, out=None) == OK
    assert attn(lib, R=0, qs=None) == OK


def test_attention_takes_the_padding_flag_with_either_type(lib):
    for kind in (0, 1):
        assert attn(lib, od=kind | 16, T=0, q=None, out=None) == OK and attn(lib, od=kind | 16, nws=100) == ESIZE
    for od in (16 | 2, 16 | 32, 32, -1, -16):
        assert attn(lib, od=od) == EINVAL, od


def test_attention_workspace_bytes(lib):
    f = lib.paged_attention_workspace_bytes
    assert f(4, 2, 4, 3, 128, 1, 10) == 0 and f(4, 2, 4, 2, 96, 1, 10) == 0
    assert 0 < f(4, 2, 4, 2, 64, 1, 10) < f(4, 2, 4, 2, 256, 1, 10)
    assert f(64, 64, 40, 8, 128, 1, 100) == f(64, 64, 40, 8, 128, 1, 10 ** 9) < 64 << 20      # independent of the lengths
    assert f(8192, 1, 40, 8, 128, 8192, 8192) == f(8192, 1, 40, 8, 128, 8192, 10 ** 9) < 128 << 20


def test_a_workspace_serves_smaller_steps(lib):
    f, g = lib.paged_attention_workspace_bytes, lib.verify_drafts_workspace_bytes
    for hq, hkv, dim in ((40, 8, 128), (24, 4, 256), (64, 1, 64)):
        for new in (1, 16, 512):
            sizes = [f(t, 64, hq, hkv, dim, new, 5000) for t in (1, 64, 300, 2000, 64 * new)]
            assert max(sizes) == sizes[-1] and f(64, 7, hq, hkv, dim, new, 50) <= sizes[-1]
    for vocab in (1, 8193, 131072, 1 << 20):
        for drafts in (0, 1, 4, 7):
            sizes = [g(r, drafts, vocab) for r in (1, 2, 3, 64, 100, 319, 320, 321, 511, 512, 2559, 2560, 2561, 9000)]
            assert sizes == sorted(sizes) and g(64, drafts, vocab) <= g(64, drafts + 1, vocab) <= g(64, drafts + 1, vocab + 9000)


def test_a_workspace_serves_steps_of_smaller_layers(lib):
    """The bytes rise with every size, with fewer KV heads for as many heads too."""
    f = lib.paged_attention_workspace_bytes
    for hkv in (1, 2, 4):
        for dim in (64, 128, 256):
            for new in (0, 1, 16, 33, 512):
                for requests in (1, 64, 5000):
                    sizes = [f(requests, requests, hkv * g, hkv, dim, new, 5000) for g in (1, 2, 8, 31, 32, 33, 40, 64, 100)]
                    assert sizes == sorted(sizes), (hkv, dim, new, sizes)
                    here = f(requests, requests, 32, hkv, dim, new, 5000)
                    assert f(requests, requests, 32, 2 * hkv, dim, new, 5000) <= here <= f(requests, requests, 32, hkv, 256, new, 5000)
                    assert here <= f(requests, requests, 32, hkv, dim, new + 1, 5000) and here <= f(requests, requests + 1, 32, hkv, dim, new, 5000)
    assert attn(lib, hq=8, heads=1, R=64, mn=16, ldq=1024, ldo=1024, nws=f(4, 64, 40, 1, 128, 16, 100)) == EHIP   # no GPU here, but bytes enough


def verify(lib, x=A16, dt=1, ldx=100, rows=6, V=100, rs=A16, nd=A16, R=2, K=2, d=A16, q=None, ldq=100, t=None, u=A16, e=A16,
           lde=100, tok=A16, acc=A16, lp=A16, ws=A16, nws=None):
    if nws is None:
        nws = lib.verify_drafts_workspace_bytes(R, K, V)
    return lib.verify_drafts(x, dt, ldx, rows, V, rs, nd, R, K, d, q, ldq, t, u, e, lde, tok, acc, lp, ws, nws, None)


def test_verify_validation(lib):
    for bad in (dict(R=-1), dict(K=-1), dict(V=0), dict(ldx=99), dict(lde=99), dict(q=A16, ldq=99), dict(rows=-1)):
        assert verify(lib, **bad) == ESHAPE, bad
    for bad in (dict(R=65536), dict(K=256), dict(V=2 ** 31 - 1)):
        assert verify(lib, **bad) == EUNSUPPORTED, bad
    for bad in (dict(x=None), dict(rs=None), dict(nd=None), dict(d=None), dict(u=None), dict(e=None), dict(tok=None),
                dict(acc=None), dict(lp=None), dict(ws=None), dict(dt=4)):
        assert verify(lib, **bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(e=0x10008), dict(q=0x10004), dict(t=MIS), dict(ws=0x10008), dict(u=MIS)):
        assert verify(lib, **bad) == EALIGN, bad
    assert verify(lib, nws=8) == ESIZE
    assert verify(lib, R=0, x=None, rs=None) == OK


def test_serving_abi_layer_under_address_and_ub_sanitizers(tmp_path):
    """abi_serving.cpp and validate_serving.cpp built for the host alone with ASan and UBSan, launchers stubbed."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "nvfp4_w4a4_gemm_quantize_amd", "csrc")
    exe = str(tmp_path / "serving_host_check")
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           os.path.join(root, "tests", "serving_host_check.cpp"), os.path.join(csrc, "abi_serving.cpp"),
           os.path.join(csrc, "validate_serving.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "cases ok" in r.stdout, r.stdout + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-4000:]


def test_binding_refuses_cpu_tensors():
    import torch
    x, i = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros((2, 1, 16, 128), dtype=torch.bfloat16)
    for call in (lambda: binding.paged_kv_write(x, x, i.long(), cache, cache),
                 lambda: binding.paged_attention(x, cache, cache, i.view(2, 2), i[:3], i[:2], 2, 8),
                 lambda: binding.paged_plan(i, i, i, i.view(4, 1), 16, 4),
                 lambda: binding.verify_drafts(x, i, i, i.view(4, 1), x, x)):
        with pytest.raises(binding.NVFP4Error):
            call()


# ------------------------------------------------------------ oracle pins --

def test_oracle_attention_closed_forms():
    """Equal keys weigh their values equally; one key gives its value; a window of one sees the token itself."""
    rng = np.random.default_rng(0)
    v = rng.standard_normal((2, 1, 16, 8))
    k = np.zeros_like(v)
    q = rng.standard_normal((3, 8))
    table, start, lens = np.array([[1, 0]]), [0, 3], [20]
    out, lse, _, _ = OP.attention(q, k, v, table, start, lens, 16, 1, 1.0)
    seq = np.concatenate([v[1, 0], v[0, 0]])
    for i in range(3):
        np.testing.assert_allclose(out[i, 0], seq[:18 + i].mean(0))
        np.testing.assert_allclose(lse[i, 0], np.log(18 + i))
    out, lse, _, _ = OP.attention(q, k, v, table, start, lens, 16, 1, 1.0, window=1)
    np.testing.assert_allclose(out[:, 0], seq[17:20])
    np.testing.assert_allclose(lse[:, 0], 0, atol=1e-12)


def test_oracle_verify_worked_example():
    """p = (1/2, 1/4, 1/4), q = (1/4, 1/2, 1/4): draft 1 is kept for u < 1/2, and the rest of p over q is word 0."""
    x = np.log(np.array([[2.0, 1, 1], [1, 1, 2]]))
    q = np.array([[[0.25, 0.5, 0.25]]])
    for u, tokens in ((0.49, [1, 2]), (0.51, [0, -1])):
        t, a, lp = OP.verify(x, [0], [1], np.array([[1]]), np.array([[u]]), np.array([[1.0, 1.0, 1.0]]), q)
        assert t.tolist() == [tokens] and a[0] == (u < 0.5)
        np.testing.assert_allclose(lp[0, 0], np.log(0.25 if u < 0.5 else 0.5))


def test_oracle_plan_worked_example():
    t, qs, sl, pos, slots, counts = OP.plan(np.array([15, 0]), np.array([2, 1]), np.array([7, 9]), 0, np.array([[3, -1], [-1, -1]]), 16, 4)
    assert t.tolist() == [[3, 7], [9, -1]] and qs.tolist() == [0, 2, 3] and sl.tolist() == [17, 1]
    assert pos.tolist() == [15, 16, 0, -1] and slots.tolist() == [63, 112, 144, -1] and counts.tolist() == [3, 2, 0, 2]
