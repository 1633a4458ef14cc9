"""Refusals of the paged-cache calls and the append's unit map, on the CPU: nothing here launches a kernel."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import libmasw_fixture  # noqa: F401
from compressed_draft_kv_gb300 import capi

HERE = os.path.dirname(os.path.abspath(__file__))


def cache(**kw):
    f = dict(k=4096, v=8192, k_scale=0, v_scale=0, page_table=256, page_stride=0, dtype=capi.MASW_BF16, n_pages=10, page_size=64,
             n_kv_heads=2, head_dim=128, batch=3, table_stride=5)
    f.update(kw)
    return capi.masw_paged_t(*[f[n] for n, _ in capi.masw_paged_t._fields_])


BAD_CACHES = [dict(dtype=0), dict(dtype=3), dict(head_dim=96), dict(page_size=48), dict(page_size=8), dict(page_size=512), dict(batch=0),
              dict(batch=513), dict(n_pages=0), dict(n_kv_heads=0), dict(table_stride=0), dict(table_stride=1 << 30), dict(k=0),
              dict(v=0), dict(page_table=0), dict(k=4100), dict(page_table=258), dict(dtype=2), dict(dtype=2, k_scale=64),
              dict(page_stride=100), dict(page_stride=64 * 2 * 128 + 4), dict(page_stride=1 << 60)]


def append(c, rows=6, kv_len=16, row_start=32, k=64, v=64, ks=0, vs=0, rope=None, pos=0, q=0, q_out=0, hq=0, qs=0, status=0):
    return capi.load().masw_paged_append(ctypes.byref(c) if c else None, kv_len, row_start, rows, k, v, ks, vs,
                                         ctypes.byref(rope) if rope else None, pos, q, q_out, hq, qs, status, None)


def attn(c, rows=6, max_rows=3, kv_len=16, row_start=32, q=64, hq=8, qs=0, window=0, scale=0.0, o=64, dt=1, lse=0, status=0, ws=64,
         wsb=1 << 40):
    return capi.load().masw_paged_attn(ctypes.byref(c) if c else None, kv_len, row_start, rows, max_rows, q, hq, qs, window, scale,
                                       o, dt, lse, status, ws, wsb, None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches_are_refused(kw):
    assert append(cache(**kw)) == capi.MASW_EINVAL
    assert attn(cache(**kw)) == capi.MASW_EINVAL
    n = ctypes.c_size_t()
    assert capi.load().masw_paged_workspace_bytes(ctypes.byref(cache(**kw)), 6, 3, 8, ctypes.byref(n)) == capi.MASW_EINVAL
    assert capi.masw_last_error()


def rope(cs=64, n=10, rot=128, inter=0):
    return capi.masw_rope_t(cs, n, rot, inter)


@pytest.mark.parametrize("kw", [
    dict(c=None), dict(rows=-1), dict(rows=7, row_start=0), dict(kv_len=0), dict(k=0), dict(v=0), dict(k=72), dict(v=72), dict(ks=128),
    dict(ks=260), dict(vs=8), dict(kv_len=18), dict(row_start=34), dict(pos=2), dict(status=2), dict(q=64, hq=4),
    dict(q=64, q_out=128), dict(q=64, q_out=128, hq=70000), dict(q=64, q_out=136, hq=4), dict(q=64, q_out=128, hq=4, qs=500),
    dict(q=64, q_out=128, hq=4, qs=516), dict(q=64, q_out=64, hq=4, qs=1024), dict(rope=rope(cs=0)), dict(rope=rope(n=0)),
    dict(rope=rope(rot=8)), dict(rope=rope(rot=40)), dict(rope=rope(rot=144)), dict(rope=rope(cs=72))])
def test_append_refusals(kw):
    kw = dict(kw)
    assert append(kw.pop("c", cache()), **kw) == capi.MASW_EINVAL
    assert "paged_append" in capi.masw_last_error()


@pytest.mark.parametrize("kw", [
    dict(c=None), dict(rows=-1), dict(rows=7, row_start=0), dict(max_rows=-1), dict(kv_len=0), dict(q=0), dict(o=0), dict(ws=0),
    dict(q=72), dict(o=72), dict(ws=72), dict(kv_len=18), dict(row_start=34), dict(lse=2), dict(status=2), dict(hq=7), dict(hq=0),
    dict(hq=2 * 129), dict(qs=1000), dict(qs=1028), dict(window=-1), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(dt=2), dict(wsb=0)])
def test_attention_refusals(kw):
    kw = dict(kw)
    rc = attn(kw.pop("c", cache()), **kw)
    assert rc == capi.MASW_EINVAL
    assert "paged" in capi.masw_last_error()


def test_nothing_to_do_is_no_error():
    assert append(cache(), rows=0) == capi.MASW_OK


def test_binding_refusals():
    k, table = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32)
    f8, sc = k.to(torch.float8_e4m3fn), torch.ones(4, 2)
    ok = capi.masw_paged_cache(k, k, table)
    assert (ok.dtype, ok.page_size, ok.batch, ok.table_stride) == (capi.MASW_BF16, 16, 2, 3)
    for bad in (lambda: capi.masw_paged_cache(k.float(), k.float(), table), lambda: capi.masw_paged_cache(k, k[:3], table),
                lambda: capi.masw_paged_cache(f8, f8, table), lambda: capi.masw_paged_cache(k, k, table, sc, sc),
                lambda: capi.masw_paged_cache(f8, f8, table, sc.double(), sc), lambda: capi.masw_paged_cache(k, k, table.long()),
                lambda: capi.masw_paged_cache(k.transpose(1, 2), k.transpose(1, 2), table),
                lambda: capi.masw_rope(torch.zeros(4, 64, dtype=torch.float64))):
        with pytest.raises(ValueError):
            bad()
    x, n = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(kv_len=n.long()), dict(kv_len=n[:1]), dict(k=x.float()), dict(k=x[:, :1]), dict(v=x[:3]), dict(q=x),
               dict(q=x, q_out=x[:3]), dict(row_start=n), dict(pos=n), dict(status=n.float())):
        a = dict(kv_len=n, k=x, v=x) | kw
        with pytest.raises(ValueError):
            capi.masw_paged_append(ok, stream=0, **a)
    o = torch.zeros(4, 2, 64)
    for kw in (dict(o=o.half()), dict(o=o[:3]), dict(lse=torch.zeros(4)), dict(q=x.float()), dict(kv_len=n.long())):
        a = dict(kv_len=n, q=x, o=o) | kw
        with pytest.raises(ValueError):
            capi.masw_paged_attn(ok, stream=0, workspace=torch.zeros(16, dtype=torch.uint8), **a)


def test_binding_refuses_what_would_be_read_out_of_range():
    """Broadcast rows and pages, whose stride of 0 would read as dense, and tensors on another device."""
    k, table = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32)
    one = k[:1].expand(4, 2, 16, 64)
    with pytest.raises(ValueError):
        capi.masw_paged_cache(one, one, table)
    c = capi.masw_paged_cache(k, k, table)
    x, n = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    row, there = x[:1].expand(4, 2, 64), dict(dtype=torch.bfloat16, device="meta")
    away = capi.masw_rope(torch.zeros(4, 64))
    away.device = torch.device("meta")
    for kw in (dict(k=row), dict(v=row), dict(q=row, q_out=x), dict(q=x, q_out=torch.zeros(4, 2, 64, **there)), dict(rope=away),
               dict(k=torch.zeros(4, 2, 64, **there)), dict(kv_len=n.to("meta"))):
        with pytest.raises(ValueError):
            capi.masw_paged_append(c, stream=0, **(dict(kv_len=n, k=x, v=x) | kw))
    ws = torch.zeros(64, dtype=torch.uint8)
    for kw in (dict(q=row), dict(workspace=ws.to("meta")), dict(workspace=ws[::2]), dict(o=x.to("meta"))):
        with pytest.raises(ValueError):
            capi.masw_paged_attn(c, stream=0, **(dict(kv_len=n, q=x, o=torch.zeros_like(x), workspace=ws) | kw))


def test_unit_map_scales_and_chunks(tmp_path):
    """The append's grid covers every touched page once, the scale exponents match a search, and the lanes of a head
    cover its elements once with paired chunks."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "paged_host")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr",
                    os.path.join(HERE, "paged_host.cu"), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    got = {a: int(b) for a, b in (line.split() for line in out.strip().splitlines())}
    assert got.pop("batches") > 500 and got.pop("scales") > 1000
    assert all(v == 0 for v in got.values()), got
