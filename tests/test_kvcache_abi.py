"""The paged key/value cache library on the CPU: it loads, exports every declared symbol, and refuses bad arguments
before any HIP call, so no GPU is needed."""
import glob
import os
import subprocess
import sys

import pytest
import torch

import means_clustering_amd as km
from means_clustering_amd import kvcache

FAKE = 0x10000    # 256-byte aligned, never dereferenced: the checks fail first
ODD4, ODD2 = FAKE + 4, FAKE + 2


@pytest.fixture(scope="module")
def L():
    return kvcache.lib()


def _cache(**kw):
    d = dict(k=FAKE, v=FAKE, pages=10, page_size=16, heads=2, dim=64, k_page=2048, k_slot=128, k_head=64, v_page=2048,
             v_slot=128, v_head=64)
    d.update(kw)
    return kvcache.KVCache(**d)


def _append(L, cache=None, dt=km.KM_BF16, T=4, q=FAKE, hq=4, qs=(256, 64), k=FAKE, ks=(128, 64), v=FAKE,
            vs=(128, 64), qw=None, kw=None, eps=1e-6,
            pos=FAKE, rope=FAKE, max_pos=100, rot=64, slots=FAKE, out=FAKE + 256,
            os=(256, 64)):
    return L.kmeans_kv_append(cache or _cache(), dt, T, q, hq, *qs, k, *ks, v, *vs, qw, kw, eps, pos, rope, max_pos,
                              rot, 0, slots, out, *os, None)


def _attend(L, cache=None, dt=km.KM_BF16, q=FAKE, T=4, hq=4, qs=(256, 64), table=FAKE, R=2, width=8, stride=8,
            starts=FAKE, lens=FAKE, lw=None, lws=(0, 0), scale=0.1, window=0, max_new=4, out=FAKE, os=(256, 64),
            lse=None, ws=FAKE, nb=1 << 40):
    return L.kmeans_kv_attend(cache or _cache(), dt, q, T, hq, *qs, table, R, width, stride, starts, lens, lw, *lws,
                              scale, window, max_new, out, *os, lse, ws, nb, None)


def _tables(L, ctx=FAKE, new=FAKE, off=None, R=4, p=16, table=FAKE, width=8, stride=8, free=FAKE, nf=5, T=4, seq=FAKE,
            qs=FAKE, ps=FAKE, pos=FAKE, slots=FAKE):
    return L.kmeans_kv_tables(ctx, new, off, R, p, table, width, stride, free, nf, T, seq, qs, ps, pos, slots, None)


def _said(L):
    return L.kmeans_kv_last_error().decode()


def test_exports_every_declared_function(L):
    declared = kvcache.header_functions()
    assert declared == ["kmeans_kv_append", "kmeans_kv_attend", "kmeans_kv_attend_workspace", "kmeans_kv_last_error",
                        "kmeans_kv_tables"]
    for name in declared:
        assert hasattr(L, name), name


BAD_CACHES = [dict(dim=8), dict(dim=72), dict(dim=272), dict(heads=0), dict(pages=0), dict(page_size=8),
              dict(page_size=24), dict(page_size=1 << 21), dict(pages=1 << 27), dict(k=None), dict(k=FAKE + 8),
              dict(k_slot=68), dict(k_head=-64), dict(v_page=1 << 41)]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_caches(L, bad):
    assert _append(L, _cache(**bad)) == 1, _said(L)
    assert _said(L)
    assert _attend(L, _cache(**bad)) == 1
    assert L.kmeans_kv_attend_workspace(_cache(**bad), 4, 4, 2, 4) == 0


def test_null_cache(L):
    assert L.kmeans_kv_append(None, 1, 4, FAKE, 4, 256, 64, FAKE, 128, 64, FAKE, 128, 64, None, None, 0.0, None, None,
                              0, 0, 0, None, FAKE, 256, 64, None) == 1
    assert "NULL" in _said(L)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 31), dict(dt=7), dict(q=None), dict(q=ODD4), dict(k=None), dict(k=ODD4), dict(v=ODD2),
    dict(out=None), dict(qs=(255, 64)), dict(ks=(128, 4)), dict(vs=(-8, 64)), dict(hq=-1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(rot=24), dict(rot=80), dict(rot=-16), dict(rope=None), dict(rope=ODD4),
    dict(pos=None), dict(pos=ODD2), dict(max_pos=0), dict(rot=0), dict(qw=ODD4), dict(kw=ODD4), dict(slots=ODD2),
    dict(out=FAKE, os=(512, 64))], ids=str)
def test_append_refusals(L, bad):
    assert _append(L, **bad) == 1, _said(L)


def test_append_limits(L):
    assert _append(L, dt=km.KM_F32) == 2
    assert _append(L, T=1 << 26) == 2
    assert _append(L, T=0) == 0  # nothing to do


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 24), dict(R=-1), dict(hq=3), dict(hq=0), dict(dt=9), dict(q=None), dict(q=ODD4),
    dict(out=None), dict(qs=(250, 64)), dict(os=(256, 60)), dict(starts=None), dict(lens=None), dict(table=None),
    dict(starts=ODD2), dict(lens=ODD2), dict(table=ODD2), dict(lse=ODD2), dict(width=-1), dict(width=1 << 28),
    dict(stride=7), dict(lw=ODD4), dict(lw=FAKE, lws=(3, 4)), dict(lw=FAKE, lws=(4, -4)), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(window=-1), dict(window=1 << 31), dict(max_new=-1), dict(ws=FAKE + 16)], ids=str)
def test_attend_refusals(L, bad):
    assert _attend(L, **bad) == 1, _said(L)


def test_attend_limits_and_workspace(L):
    assert _attend(L, dt=km.KM_F32) == 2
    assert _attend(L, ws=None, nb=0) == 3
    need = L.kmeans_kv_attend_workspace(_cache(), 4, 4, 2, 4)
    assert need > 0
    assert _attend(L, nb=need - 1) == 3 and "too small" in _said(L)
    assert _attend(L, T=0) == 0 and _attend(L, R=0) == 0 and _attend(L, max_new=0) == 0  # nothing to do
    assert _attend(L, _cache(heads=1 << 14, k_page=1 << 30, v_page=1 << 30), hq=1 << 14, qs=(1 << 20, 64),
                   os=(1 << 20, 64), T=1 << 12, R=1 << 12, max_new=1) == 2
    big = L.kmeans_kv_attend_workspace(_cache(heads=8, dim=128), 1 << 14, 64, 16, 1 << 12)
    assert 0 < big < 1 << 28  # a prefill of 16,384 tokens: parts, not whole scores


@pytest.mark.parametrize("bad", [
    dict(R=-1), dict(R=1 << 24), dict(T=-1), dict(p=8), dict(p=48), dict(width=-1), dict(stride=7),
    dict(width=1 << 27, stride=1 << 27),
    dict(nf=-1), dict(qs=None), dict(ps=None), dict(ctx=None), dict(new=None), dict(seq=None), dict(table=None),
    dict(free=None), dict(pos=None), dict(slots=None), dict(ctx=ODD2), dict(off=ODD2), dict(slots=ODD2)], ids=str)
def test_tables_refusals(L, bad):
    assert _tables(L, **bad) == 1, _said(L)


def test_python_binding_rejects_host_tensors():
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        kvcache.append(None, c[0, :1], None, c, None, None)
    with pytest.raises(ValueError, match="device"):
        kvcache.attend(c[0, :1], c, c, torch.zeros(1, 2, dtype=torch.int32), i, i)
    with pytest.raises(ValueError, match="device"):
        kvcache.tables(i, i, torch.zeros(1, 2, dtype=torch.int32), i, 16, 1)


def test_checks_under_asan_ubsan(tmp_path):
    """The host side (argument checks, plans, workspace sizes) rebuilt with AddressSanitizer and
    UndefinedBehaviorSanitizer on the host, linked with the kernels' objects of the regular build, and this file's
    other tests run against it in a child process with the sanitizer runtime preloaded."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    objs = [os.path.join(root, "_build", f + ".o") for f in ("kv_tables.hip", "kv_append.hip", "kv_decode.hip",
                                                             "kv_chunk.hip")]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("needs the kernel objects of the regular build (__graft_entry__.build())")
    rts = glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    if not rts:
        pytest.skip("clang AddressSanitizer runtime not found")
    hipcc = "/opt/rocm/bin/hipcc"
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-omit-frame-pointer"]
    mine, lib = str(tmp_path / "kv_api.o"), str(tmp_path / "libkm_cache_asan.so")
    subprocess.run([hipcc, "-std=c++17", "-O1", "-g", "-fPIC", "--offload-arch=gfx950", *host_san,
                    "-I", os.path.join(root, "include"), "-c",
                    os.path.join(root, "means_clustering_amd", "csrc", "kv_api.cpp"), "-o", mine],
                   check=True, capture_output=True)
    subprocess.run([hipcc, "-shared", "-fPIC", "--offload-arch=gfx950", *host_san, "-shared-libasan", mine, *objs,
                    "-o", lib], check=True, capture_output=True)
    old = os.environ.get("LD_PRELOAD", "")
    env = dict(os.environ, LD_PRELOAD=rts[0] + (":" + old if old else ""), ASAN_OPTIONS="detect_leaks=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, os.path.join(root, "tests", "native", "run_with_cache_lib.py"), lib,
                        "-s", "-k", "not under_asan"], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
