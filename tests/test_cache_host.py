"""Host-side checks of the paged cache's C ABI (include/dspark_cache.h): symbols,
workspace sizes, refusals.  Validation runs before anything is enqueued, so no
call here needs a GPU or reaches a kernel launch."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dspark_cache.h")
GOOD = dict(B=4, n_pages=100, page=16, max_pages=10, n_layers=2, Hq=8, Hkv=2, D=128)


@pytest.fixture(scope="module")
def ds():
    from draft_sampling_verification_markov_amd import dspark
    if not os.path.exists(dspark.LIB_PATH):
        from draft_sampling_verification_markov_amd import build
        build.build()
    dspark.load()
    return dspark


@pytest.mark.parametrize("debug", [False, True], ids=["libdspark", "libdspark_debug"])
def test_library_exports_what_the_header_declares(ds, debug):
    declared = sorted(set(re.findall(r"\b(dspark_[a-z_]+)\s*\(", open(HEADER).read())))
    assert declared == sorted(ds.CACHE_SYMBOLS)
    path = ds.DEBUG_LIB_PATH if debug else ds.LIB_PATH
    out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True, check=True)
    exported = set(re.findall(r"\sT\s(dspark_\w+)", out.stdout))
    assert set(declared) <= exported


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#define __HIP_PLATFORM_AMD__ 1\n#include "dspark_cache.h"\n'
                   "int main(void) { dspark_cache c = {0}; return c.B + DSPARK_F8E4M3 - 2; }\n")
    subprocess.run(["gcc", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), "-I/opt/rocm/include", str(src)],
                   check=True)


def problem(ds, q="bf16", cache="bf16", **kw):
    return ds.Cache.make(**{**GOOD, **kw}, q=q, cache=cache)


BAD = [(dict(B=0), -1), (dict(B=65537), -1), (dict(n_pages=0), -1), (dict(n_pages=(1 << 24) + 1), -1), (dict(page=0), -1),
       (dict(page=24), -3), (dict(page=512), -3), (dict(max_pages=0), -1), (dict(max_pages=(1 << 20) + 1), -1),
       (dict(n_layers=0), -1), (dict(n_layers=1025), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(Hq=9), -1),
       (dict(Hq=2048), -1), (dict(D=0), -1), (dict(D=96), -3), (dict(D=512), -3),
       (dict(q="f32"), -3), (dict(cache="f32"), -3), (dict(q="f32", cache="f8"), -3)]


class Memory:
    """Addresses that validation accepts; nothing behind them is touched."""
    base = 1 << 40

    def __getattr__(self, name):
        a = Memory.base
        Memory.base += 1 << 32
        setattr(self, name, a)
        return a


def calls(ds, C, m, **kw):
    a = dict(layer=0, k=m.k, ks=256, v=m.v, vs=256, q=m.q, qs=1024, rows=4, n_new=m.n, row_start=m.r, max_new=3,
             length=m.length, table=m.table, k_pool=m.kp, v_pool=m.vp, k_scale=None, v_scale=None, scale=0.1, window=0,
             out=m.out, os=1024, lse=m.lse, ws=m.ws, wb=1 << 30, parent=None, new_len=m.new, ref=m.ref, to=m.to, lo=m.lo,
             ro=m.ro, count=m.count)
    a.update(kw)
    lib = ds.load()
    return {
        "append": lambda: lib.dspark_cache_append(C, a["layer"], a["k"], a["ks"], a["v"], a["vs"], a["rows"], a["n_new"],
                                                  a["row_start"], a["max_new"], a["length"], a["table"], a["k_scale"],
                                                  a["v_scale"], a["k_pool"], a["v_pool"], None),
        "attend": lambda: lib.dspark_cache_attend(C, a["layer"], a["q"], a["qs"], a["rows"], a["n_new"], a["row_start"],
                                                  a["max_new"], a["length"], a["table"], a["k_pool"], a["v_pool"],
                                                  a["k_scale"], a["v_scale"], a["scale"], 1, a["window"], a["out"],
                                                  a["os"], a["lse"], a["ws"], a["wb"], None),
        "update": lambda: lib.dspark_cache_update(C, a["parent"], a["new_len"], a["table"], a["length"], a["ref"],
                                                  a["to"], a["lo"], a["ro"], a["count"], a["k_pool"], a["v_pool"],
                                                  a["ws"], a["wb"], None),
        "compact": lambda: lib.dspark_cache_compact(C, a["table"], a["length"], a["ref"], a["to"], a["ro"], a["count"],
                                                    a["k_pool"], a["v_pool"], a["ws"], a["wb"], None),
    }


@pytest.mark.parametrize("change,status", BAD, ids=[str(b[0]) for b in BAD])
def test_bad_geometry_is_refused_by_every_call(ds, change, status):
    C = problem(ds, **change)
    assert ds.cache_workspace_bytes(C, 3) == 0
    for name, call in calls(ds, C, Memory()).items():
        assert call() == status, name


def test_bad_types_are_refused(ds):
    for field, value in (("data_dtype", 2), ("data_dtype", 9), ("cache_dtype", 3), ("cache_dtype", -1)):
        C = problem(ds)
        setattr(C, field, value)
        for name, call in calls(ds, C, Memory()).items():
            assert call() == ds.E_DTYPE, (name, field, value)


INV, PTR, WSP = -1, -6, -4
REFUSED = [
    ("append attend", dict(layer=2), INV), ("append attend", dict(layer=-1), INV), ("append attend", dict(rows=-1), INV),
    ("append attend", dict(max_new=0), INV), ("append attend", dict(max_new=(1 << 20) + 1), INV),
    ("append attend update compact", dict(length=None), PTR), ("append attend update compact", dict(table=None), PTR),
    ("append attend update compact", dict(k_pool=None), PTR), ("append attend update compact", dict(v_pool=None), PTR),
    ("append attend update compact", dict(k_pool=(1 << 41) + 8), PTR), ("append attend", dict(n_new=(1 << 41) + 2), PTR),
    ("append", dict(k=None), PTR), ("append", dict(v=(1 << 41) + 4), PTR), ("append", dict(ks=255), INV),
    ("append", dict(vs=260), INV), ("append", dict(ks=248), INV), ("attend", dict(qs=1000), INV),
    ("attend", dict(q=None), PTR), ("attend", dict(out=None), PTR), ("attend", dict(os=8), INV),
    ("attend", dict(scale=0.0), INV), ("attend", dict(scale=-1.0), INV), ("attend", dict(scale=float("inf")), INV), ("attend", dict(scale=3e38), INV),
    ("attend", dict(scale=float("nan")), INV), ("attend", dict(window=-1), INV), ("attend", dict(lse=(1 << 41) + 1), PTR),
    ("attend update compact", dict(ws=None), WSP), ("attend update compact", dict(ws=(1 << 41) + 128), WSP),
    ("attend update compact", dict(wb=64), WSP), ("update", dict(new_len=None), PTR),
    ("update compact", dict(ref=None), PTR), ("update compact", dict(to=None), PTR), ("update", dict(lo=None), PTR),
    ("update compact", dict(ro=None), PTR), ("update compact", dict(count=None), PTR),
    ("update", dict(parent=(1 << 41) + 2), PTR),
]


@pytest.mark.parametrize("names,change,status", REFUSED, ids=[f"{a.split()[0]}-{b}" for a, b, _ in REFUSED])
def test_bad_arguments_are_refused(ds, names, change, status):
    for name in names.split():
        assert calls(ds, problem(ds), Memory(), **change)[name]() == status, name


def test_outputs_over_inputs_are_refused(ds):
    for out, src in (("to", "table"), ("lo", "length"), ("ro", "ref"), ("count", "new_len"), ("lo", "new_len"),
                     ("to", "ref")):
        m = Memory()
        assert calls(ds, problem(ds), m, **{out: getattr(m, "new" if src == "new_len" else src)})["update"]() == PTR
    for out, src in (("to", "table"), ("ro", "ref"), ("count", "length")):
        m = Memory()
        assert calls(ds, problem(ds), m, **{out: getattr(m, src)})["compact"]() == PTR


def test_e4m3_needs_its_scales(ds):
    C = problem(ds, cache="f8")
    m = Memory()
    for kw in (dict(), dict(k_scale=m.s), dict(v_scale=m.s), dict(k_scale=m.s + 2, v_scale=m.s)):
        c = calls(ds, C, m, **kw)
        assert c["append"]() == PTR and c["attend"]() == PTR


def test_more_row_tiles_than_attend_serves(ds):
    # 65536 requests x 2^20 rows x 1024 heads of a group: refused, not searched for hours
    C = problem(ds, B=65536, Hq=1024, Hkv=1)
    assert calls(ds, C, Memory(), max_new=1 << 20, qs=1024 * 128, os=1024 * 128)["attend"]() == INV
    C = problem(ds, B=4096, Hq=16, Hkv=1)
    assert calls(ds, C, Memory(), max_new=4097, qs=2048, os=2048)["attend"]() == INV


def test_null_cache_and_no_rows(ds):
    for name, call in calls(ds, None, Memory()).items():
        assert call() == PTR, name
    c = calls(ds, problem(ds), Memory(), rows=0, q=None, out=None, k=None, v=None)
    assert c["append"]() == ds.OK and c["attend"]() == ds.OK


def test_workspace_sizes(ds):
    a = ds.cache_workspace_bytes(problem(ds), 1)
    assert a > 0 and a % 256 == 0
    assert ds.cache_workspace_bytes(problem(ds), 0) == 0
    assert ds.cache_workspace_bytes(problem(ds), (1 << 20) + 1) == 0
    assert ds.cache_workspace_bytes(problem(ds, n_pages=1 << 23), 1) > a


def test_binding_refuses_host_tensors(ds):
    import torch
    C = problem(ds)
    x = torch.zeros(1)
    with pytest.raises(ValueError, match="device"):
        ds.cache_append(C, 0, x, x, None, None, 1, x, x, None, None, x, x)
