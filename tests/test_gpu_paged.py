"""Paged-cache operators on the GPU against the fp64 oracle: append with rotation, attention, and both as a
speculative step uses them."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as po
from compressed_draft_kv_gb300 import capi
from paged_helpers import DEV, E4M3, Cache, check_attention, ints, np64, starts, tables

pytestmark = pytest.mark.gpu


def bf16(*shape, seed=0, mul=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * mul).to(torch.bfloat16).to(DEV)


# ------------------------------------------------------------------ append --

def run_append(c, kv, n, hq, seed=0, rot=None, inter=False, strided=False, pos=None, first=0, pad=0, mul=1.0, edit=None,
               n_pos=2048, uniform=False):
    """One append checked bit for bit: pages, scales and rotated q; rows that are padding stay."""
    rs = starts(n, first)
    T = rs[-1] + pad
    hkv, d = c.hkv, c.d
    fused = bf16(T, (hq + 2 * hkv) * d, seed=seed, mul=mul)
    if edit is not None:
        edit(fused)
    q, k, v = fused[:, :hq * d], fused[:, hq * d:(hq + hkv) * d], fused[:, (hq + hkv) * d:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q, k, v = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
    cs = None if rot is None else tables(n_pos, rot)
    rope = None if rot is None else capi.masw_rope(cs.to(DEV), inter)
    q_out = torch.full((T, hq, d), 3.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = c.mirror()
    dense_q = q.contiguous()
    capi.masw_paged_append(c.c, ints(kv), k, v, rope=rope, pos=None if pos is None else ints(pos), q=q, q_out=q_out,
                           row_start=None if uniform else ints(rs), status=status)
    torch.cuda.synchronize()
    wq = po.append(want, c.table.tolist(), kv, rs, np64(k), np64(v), None if cs is None else cs.numpy(), inter, pos, np64(dense_q))
    assert status.item() == 0
    got = c.mirror()
    for name in ("k_scale", "v_scale", "k", "v"):
        if want[name] is not None:
            assert np.array_equal(got[name], want[name], equal_nan=True), name
    real = slice(rs[0], rs[-1])
    assert np.array_equal(np64(q_out)[real], wq[real], equal_nan=True)
    assert (q_out[:rs[0]] == 3.0).all() and (q_out[rs[-1]:] == 3.0).all()
    return got


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,page,hkv,hq,rot,inter,strided", [
    (128, 64, 2, 6, 128, False, True), (128, 16, 1, 5, 32, True, False), (64, 32, 3, 3, 64, True, True),
    (64, 128, 2, 2, 16, False, False), (128, 256, 1, 1, None, False, True)])
def test_append_rows_of_every_kind(dtype, d, page, hkv, hq, rot, inter, strided):
    n = [1, 0, 3, page, 1, page + 5, 2 * page + 1]
    before = [0, 9, page - 1, 5, 2 * page, page - 3, 0]       # starts a page, ends inside, crosses, fills exactly
    kv = [a + b for a, b in zip(n, before)]
    c = Cache(kv, hkv, d, page, dtype, seed=d + page)
    run_append(c, kv, n, hq, seed=1, rot=rot, inter=inter, strided=strided)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_padded_batch_and_pages_apart(dtype):
    n, kv = [4, 0, 17], [30, 12, 17]
    c = Cache(kv, 2, 128, 16, dtype, seed=3, gap=1)
    run_append(c, kv, n, 4, seed=2, rot=64, first=5, pad=7)


@pytest.mark.parametrize("rows", [1, 3])
def test_append_uniform_rows_and_own_positions(rows):
    kv = [20, 21, 35]
    c = Cache(kv, 2, 64, 32, "e4m3", seed=4)
    run_append(c, kv, [rows] * 3, 2, seed=3, rot=64, pos=[(7 * i + 3) % 50 for i in range(3 * rows)], n_pos=50, uniform=True)


def test_append_scale_grows_by_powers_of_two_and_never_shrinks_in_a_page():
    """Token after token with growing, then shrinking, then zero rows: the page's rows are rounded again at each growth;
    a page whose first row is zero starts at scale 1; a rejected draft's rows are overwritten."""
    c = Cache([70], 2, 64, 32, "e4m3", seed=5)
    lengths = list(range(1, 40)) + [36, 37, 64, 65]
    prev = 0
    for i, kv in enumerate(lengths):
        n = kv - prev if kv > prev else 2
        mul = 0.0 if kv in (33, 34) else 2.0 ** ((i * 5) % 11 - 5)
        run_append(c, [kv], [n], 1, seed=i, rot=64, mul=mul)
        prev = kv


def test_append_borders_of_the_scale_and_of_the_type():
    """amax exactly at 448 times a power of two, just above it, ties, subnormals, the smallest and largest scales."""
    c = Cache([32] * 6, 1, 64, 32, "e4m3", seed=6)

    def edit(x):
        x[0:2] = 1.75 * 2.0 ** 3                # exactly 448 * 2^-5
        x[2:4] = 1.7578125 * 2.0 ** 3           # the next bf16
        x[4:6, 0::2], x[4:6, 1::2] = 448.0, 17.0    # 17 / 1: a tie between 16 and 18
        x[6:8, 1::2] = x[6:8, 1::2] * 1e-4      # subnormals beside ordinary values
        x[8:10] = 1e-30                         # below the smallest scale
        x[10:12] = 3e38 * torch.sign(x[10:12].float()).to(x.dtype)

    with np.errstate(over="ignore"):
        run_append(c, [2] * 6, [2] * 6, 1, seed=7, rot=None, edit=edit)


def test_append_keeps_what_is_not_finite_apart():
    """Infinities and NaN become NaN, and the scale of their page and head covers the finite rest."""
    c = Cache([40, 40], 2, 64, 16, "e4m3", seed=8)

    def edit(x):
        x[3, 5], x[3, 70], x[9, 130], x[9, 64 * 3 + 2] = float("inf"), float("nan"), float("-inf"), float("nan")
        x[14, :] = float("nan")                 # nothing finite in a row of every head

    run_append(c, [12, 19], [12, 3], 1, seed=9, rot=None, edit=edit)


def test_append_reports_bad_lengths_rows_pages_and_positions_and_skips_them():
    kv, n = [20, 10, 33], [4, 2, 3]
    for what in ("page", "page_negative", "length", "short", "rows", "backwards", "position"):
        c = Cache(kv, 1, 64, 16, "e4m3", seed=10)
        table, kvl, rs, pos = c.table.clone(), list(kv), starts(n), list(range(9))
        if what == "page":
            table[1, 0] = c.k.shape[0]
        elif what == "page_negative":
            table[1, 0] = -1
        elif what == "length":
            kvl[1] = table.shape[1] * 16 + 1
        elif what == "short":
            kvl[1] = 1                          # fewer than its rows
        elif what == "rows":
            rs[3] = 10                          # more than there are
        elif what == "backwards":
            rs[1], rs[2] = 6, 4
        else:
            pos[5] = 64
        table = table.to(DEV)
        cc = capi.masw_paged_cache(c.k, c.v, table, c.ks, c.vs)
        k, v, q = bf16(9, 1, 64), bf16(9, 1, 64, seed=1), bf16(9, 2, 64, seed=2)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        before = c.mirror()
        capi.masw_paged_append(cc, ints(kvl), k, v, rope=capi.masw_rope(tables(64, 64).to(DEV)), pos=ints(pos), q=q,
                               q_out=torch.empty_like(q), row_start=ints(rs), status=status)
        torch.cuda.synchronize()
        assert status.item() == capi.MASW_EINVAL, what
        got = c.mirror()
        touched = {int(p) for b in range(3) for p in c.table[b] if p >= 0}
        spare = [i for i in range(c.k.shape[0]) if i not in touched]
        assert np.array_equal(got["k"][spare], before["k"][spare]), what
        if what in ("page", "page_negative", "length", "short"):      # the other sequences are served
            want = before
            po.append(want, c.table.tolist(), [20, 0, 33], [0, 4, 4, 7], np64(k)[[0, 1, 2, 3, 6, 7, 8]],
                      np64(v)[[0, 1, 2, 3, 6, 7, 8]], tables(64, 64).numpy(), False, [0, 1, 2, 3, 6, 7, 8])
            assert np.array_equal(got["k"], want["k"]) and np.array_equal(got["v_scale"], want["v_scale"]), what


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,page,rot,inter", [(128, 256, 128, False), (64, 128, 32, True), (128, 128, None, False)])
def test_append_few_rows_on_large_pages(dtype, d, page, rot, inter):
    """Steps: pages far from full, page borders inside the rows, more rows than one pass over them holds."""
    n = [1, 5, 0, 4, 2, 9]
    kv = [7, page + 2, 3, page, 2 * page + 1, 2 * page + 8]
    c = Cache(kv, 3, d, page, dtype, seed=d + page + 1)
    run_append(c, kv, n, 5, seed=11, rot=rot, inter=inter, strided=True)


@pytest.mark.parametrize("rows", [1, 2, 6])
def test_append_uniform_steps_on_large_pages(rows):
    kv = [20, 257, 256, 6, 130]
    c = Cache(kv, 2, 128, 256, "e4m3", seed=12)
    run_append(c, kv, [rows] * 5, 3, seed=13, rot=128, uniform=True, strided=True)


@pytest.mark.parametrize("rows", [1, 2, 9])
def test_append_of_a_large_batch(rows):
    kv = [rows + (37 * b) % 60 for b in range(300)]
    c = Cache(kv, 4, 64, 64, "e4m3", seed=14)
    run_append(c, kv, [rows] * 300, 8, seed=15, rot=64)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,hkv,hq", [(128, 7, 57), (256, 5, 33)])
def test_append_of_a_prompt_with_many_heads(dtype, page, hkv, hq):
    """A CTA takes several heads in turn, K, V and Q among them; the last group is not full."""
    n, kv = [2500, 1301], [2507, 1301]
    c = Cache(kv, hkv, 128, page, dtype, seed=16)
    run_append(c, kv, n, hq, seed=17, rot=96, strided=True, n_pos=4096)


@pytest.mark.parametrize("page", [128, 256])
def test_append_steps_report_what_is_bad_and_skip_it(page):
    kv, n = [20, 10, 33], [4, 2, 3]
    for what in ("page", "length", "short", "rows", "position"):
        c = Cache(kv, 1, 64, page, "e4m3", seed=18)
        table, kvl, rs, pos = c.table.clone(), list(kv), starts(n), list(range(9))
        if what == "page":
            table[1, 0] = c.k.shape[0]
        elif what == "length":
            kvl[1] = table.shape[1] * page + 1
        elif what == "short":
            kvl[1] = 1
        elif what == "rows":
            rs[3] = 10
        else:
            pos[5] = 64
        cc = capi.masw_paged_cache(c.k, c.v, table.to(DEV), c.ks, c.vs)
        k, v = bf16(9, 1, 64, seed=19), bf16(9, 1, 64, seed=20)
        before, status = c.mirror(), torch.zeros(1, dtype=torch.int32, device=DEV)
        rope = capi.masw_rope(tables(64, 64).to(DEV))
        capi.masw_paged_append(cc, ints(kvl), k, v, rope=rope, pos=ints(pos), row_start=ints(rs), status=status)
        torch.cuda.synchronize()
        assert status.item() == capi.MASW_EINVAL
        after, hit = c.mirror(), int(c.table[2 if what == "rows" else 1, 0])
        changed = {p for name in before for p in np.argwhere(after[name] != before[name])[:, 0].tolist()}
        assert changed == {int(c.table[b, 0]) for b in range(3)} - (set() if what == "position" else {hit})


def test_append_in_place_q_and_no_q():
    c = Cache([5, 40], 2, 128, 16, "bf16", seed=11)
    k, v, q = bf16(5, 2, 128), bf16(5, 2, 128, seed=1), bf16(5, 4, 128, seed=2)
    q0 = np64(q)
    cs = tables(64, 128)
    want = c.mirror()
    rope = capi.masw_rope(cs.to(DEV))
    capi.masw_paged_append(c.c, ints([5, 40]), k, v, rope=rope, q=q, q_out=q, row_start=ints([0, 2, 5]))
    wq = po.append(want, c.table.tolist(), [5, 40], [0, 2, 5], np64(k), np64(v), cs.numpy(), False, None, q0)
    assert np.array_equal(np64(q), wq)
    first = c.mirror()
    assert np.array_equal(first["k"], want["k"])
    capi.masw_paged_append(c.c, ints([5, 40]), k, v, rope=rope, row_start=ints([0, 2, 5]))
    assert np.array_equal(c.mirror()["k"], want["k"]) and np.array_equal(c.mirror()["v"], want["v"])


def test_append_at_large_offsets():
    """Pages whose byte offsets pass 32 bits."""
    page, hkv, d = 256, 8, 128
    far = (1 << 32) // (page * hkv * d) + 3
    c = Cache([300], hkv, d, page, "e4m3", seed=12, fill=False, first_page=far)
    used = [int(p) for p in c.table[0] if p >= 0]
    c.k[used], c.v[used] = 0, 0
    k, v = bf16(300, hkv, d), bf16(300, hkv, d, seed=1)
    capi.masw_paged_append(c.c, ints([300]), k, v)
    small = {"k": np.zeros((len(used), hkv, page, d)), "v": np.zeros((len(used), hkv, page, d)),
             "k_scale": np.ones((len(used), hkv)), "v_scale": np.ones((len(used), hkv))}
    po.append(small, [list(range(len(used)))], [300], [0, 300], np64(k), np64(v))
    assert np.array_equal(np64(c.k[used].view(E4M3)), small["k"]) and np.array_equal(np64(c.v[used].view(E4M3)), small["v"])
    assert np.array_equal(np64(c.ks[used]), small["k_scale"])
    q, o, lse = bf16(2, 16, d, seed=3), torch.empty(2, 16, d, dtype=torch.bfloat16, device=DEV), torch.empty(2, 16, device=DEV)
    capi.masw_paged_attn(c.c, ints([300]), q, o, lse)
    check_attention(small, [list(range(len(used)))], [300], [0, 2], q, o, lse)


# --------------------------------------------------------------- attention --

def run_attention(c, kv, n, hq, seed=0, window=0, scale=0.0, o_dtype=torch.bfloat16, first=0, pad=0, strided=False, mul=1.0,
                  max_rows=None, uniform=False, q=None):
    rs = starts(n, first)
    T = rs[-1] + pad
    if q is None:
        q = bf16(T, hq, 2 * c.d if strided else c.d, seed=seed, mul=mul)
        if strided:
            q = q.reshape(T, 2 * hq, c.d)[:, :hq]
    o = torch.full((T, hq, c.d), 3.0, dtype=o_dtype, device=DEV)
    lse = torch.full((T, hq), 3.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    capi.masw_paged_attn(c.c, ints(kv), q, o, lse, row_start=None if uniform else ints(rs), max_rows=max_rows or max(n),
                         window=window, scale=scale, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    check_attention(c.mirror(), c.table.tolist(), kv, rs, q, o, lse, window, scale or None)
    assert (o[:rs[0]] == 3.0).all() and (o[rs[-1]:] == 3.0).all() and (lse[rs[-1]:] == 3.0).all()
    return o, lse


KINDS = [(d, e) for d in (128, 64) for e in ("bf16", "e4m3")]


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("hkv,g,page", [(2, 4, 64), (1, 3, 16), (3, 1, 32), (1, 8, 256), (2, 5, 128), (1, 32, 32)])
def test_decode_ragged_lengths(d, dtype, hkv, g, page):
    kv = [1, 2, 127, 128, 129, 300, 16, 257]
    run_attention(Cache(kv, hkv, d, page, dtype, seed=g + page), kv, [1] * 8, hkv * g, seed=g, uniform=page == 16)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("hkv,g,page,o_dtype", [(2, 4, 64, torch.bfloat16), (1, 3, 16, torch.float32), (2, 1, 32, torch.bfloat16)])
def test_few_rows_ragged(d, dtype, hkv, g, page, o_dtype):
    n, kv = [1, 6, 0, 3, 7, 2], [70, 6, 50, 131, 600, 2]
    run_attention(Cache(kv, hkv, d, page, dtype, seed=g), kv, n, hkv * g, seed=g + 1, o_dtype=o_dtype, first=2, pad=3, strided=True)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("hkv,g,page", [(1, 4, 64), (2, 3, 16), (1, 1, 128), (1, 6, 32), (1, 40, 64)])
def test_long_blocks_ragged(d, dtype, hkv, g, page):
    n, kv = [90, 1, 0, 33, 128], [90, 500, 10, 300, 129]
    run_attention(Cache(kv, hkv, d, page, dtype, seed=g), kv, n, hkv * g, seed=g + 2, first=1, pad=2, strided=g == 3)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("n,kv,g,page,window,o_dtype", [
    ([9, 16, 17], [9, 200, 385], 4, 64, 0, torch.bfloat16), ([33, 20, 1], [2001, 129, 1], 2, 16, 0, torch.float32),
    ([32, 31, 9], [1500, 31, 256], 4, 32, 100, torch.bfloat16), ([16, 1, 12], [4000, 128, 700], 8, 128, 300, torch.float32),
    ([90, 64, 50], [640, 64, 300], 1, 64, 0, torch.bfloat16)])
def test_blocks_of_one_tile_of_rows(d, dtype, n, kv, g, page, window, o_dtype):
    """More rows than the few-rows kernel takes and at most 128: one tile, or two where a sequence has more."""
    c = Cache(kv, 2, d, page, dtype, seed=62)
    run_attention(c, kv, n, 2 * g, seed=63, window=window, o_dtype=o_dtype, pad=2)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("n,window", [([1, 1, 1], 1), ([1, 1, 1], 100), ([3, 2, 8], 128), ([3, 2, 8], 5), ([150, 40, 1], 64),
                                      ([150, 40, 1], 129), ([150, 40, 1], 100000)])
def test_sliding_window(d, dtype, n, window):
    kv = [400, 129, 77]
    run_attention(Cache(kv, 1, d, 32, dtype, seed=window), kv, n, 4, seed=window, window=window)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("n,kv", [([1, 1, 2], [0, 5, 0]), ([4, 3, 6], [2, 0, 6]), ([50, 60, 70], [20, 0, 70])])
def test_rows_that_see_nothing(d, dtype, n, kv):
    run_attention(Cache([max(1, x) for x in kv], 1, d, 16, dtype, seed=1), kv, n, 4, seed=2)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("n", [[1, 1], [3, 5], [45, 70]])
def test_nan_behind_the_end_and_outside_the_window(d, dtype, n):
    """Rows behind a sequence's end, whole unused pages and (for one query row) keys before the window hold NaN."""
    kv = [77, 150]
    c = Cache(kv, 2, d, 32, dtype, seed=3)
    window = 40 if n == [1, 1] else 0
    bad = 0x7F if c.e4 else float("nan")
    used = set()
    for b in range(2):
        for p in range(kv[b]):
            used.add((int(c.table[b, p // 32]), p % 32))
            if window and p < kv[b] - window:
                c.k[int(c.table[b, p // 32]), :, p % 32] = bad
                c.v[int(c.table[b, p // 32]), :, p % 32] = bad
    for pid in range(c.k.shape[0]):
        for r in range(32):
            if (pid, r) not in used:
                c.k[pid, :, r], c.v[pid, :, r] = bad, bad
        if c.e4 and not any((pid, r) in used for r in range(32)):
            c.ks[pid], c.vs[pid] = float("nan"), float("nan")
    o, lse = run_attention(c, kv, n, 4, seed=4, window=window)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("n", [[1, 1], [4, 6], [60, 33]])
def test_large_and_small_scores(d, dtype, n):
    """Peaked softmax, scores far from zero, maxima that keep rising along the cache, scale given by the caller."""
    kv = [513, 290]
    c = Cache(kv, 1, d, 32, dtype, seed=5)
    run_attention(c, kv, n, 3, seed=6, mul=6.0)
    run_attention(c, kv, n, 3, seed=7, mul=1e-3, scale=0.7)
    if c.e4:
        order = [int(p) for p in c.table[0] if p >= 0]
        c.ks[order, 0] = torch.exp2(torch.linspace(-14, -3, len(order), device=DEV).round())
    else:
        order = [int(p) for p in c.table[0] if p >= 0]
        c.k[order] *= torch.exp2(torch.linspace(-9, 1, len(order), device=DEV).round()).to(torch.bfloat16)[:, None, None, None]
    run_attention(c, kv, n, 3, seed=8)


@pytest.mark.parametrize("n", [[1], [5], [70]])
def test_v_scales_of_very_different_size_and_not_powers_of_two(n):
    c = Cache([700], 2, 128, 64, "e4m3", seed=9)
    order = [int(p) for p in c.table[0] if p >= 0]
    c.vs[order, 0] = 2.0 ** -60
    c.vs[order[3:5], 0] = 2.0 ** 40
    c.vs[order, 1] = torch.rand(len(order), device=DEV) * 3e-3 + 1e-5
    c.ks[order, 1] = torch.rand(len(order), device=DEV) * 1e-2 + 1e-3
    run_attention(c, [700], n, 8, seed=10)


@pytest.mark.parametrize("d,dtype", KINDS)
@pytest.mark.parametrize("n,hkv,g,page,window", [(1, 8, 4, 16, 0), (6, 8, 4, 64, 0), (1, 2, 8, 32, 1000)])
def test_a_serving_batch_repeats_bit_for_bit(d, dtype, n, hkv, g, page, window):
    """Every SM streams several sequences one behind the other, the values' stream behind the keys'."""
    kv = [700 + (911 * b) % 2900 for b in range(32)]
    c = Cache(kv, hkv, d, page, dtype, seed=60)
    o, lse = run_attention(c, kv, [n] * 32, hkv * g, seed=61, window=window, uniform=True)
    q = bf16(32 * n, hkv * g, d, seed=61)
    for _ in range(20):
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        capi.masw_paged_attn(c.c, ints(kv), q, o2, lse2, window=window)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_many_sequences_split_and_whole(dtype):
    """Short sequences beside long ones, one kv head: some are cut over many CTAs, some share one."""
    g = np.random.default_rng(1)
    kv = [int(x) for x in g.integers(1, 90, 60)] + [5000] + [int(x) for x in g.integers(1, 400, 20)]
    c = Cache(kv, 1, 64, 16, dtype, seed=11)
    run_attention(c, kv, [1] * len(kv), 2, seed=12)
    n = [int(x) for x in g.integers(0, 5, len(kv))]
    run_attention(c, kv, n, 2, seed=13)


def test_non_finite_values_that_rows_see():
    """A NaN or an infinity in a visible key or value reaches the rows that see it; the same call's other sequences do
    not notice."""
    c = Cache([64, 64], 1, 128, 32, "bf16", seed=14)
    c.k[int(c.table[0, 0]), 0, 3, 5] = float("nan")
    q = bf16(2, 4, 128, seed=1)
    o, lse = torch.empty_like(q), torch.empty(2, 4, device=DEV)
    capi.masw_paged_attn(c.c, ints([64, 64]), q, o, lse)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all() and torch.isfinite(o[1]).all()


def test_attention_reports_bad_pages_lengths_and_rows():
    kv, n = [200, 100, 40], [3, 2, 1]
    for rows in (n, [80, 2, 1]):
        for what in ("page", "page_negative", "length", "rows", "backwards", "max_rows"):
            c = Cache(kv, 1, 64, 16, "e4m3", seed=10)
            table, kvl, rs, mr = c.table.clone(), list(kv), starts(rows), max(rows)
            if what == "page":
                table[1, 2] = c.k.shape[0]
            elif what == "page_negative":
                table[1, 2] = -1
            elif what == "length":
                kvl[1] = table.shape[1] * 16 + 1
            elif what == "rows":
                rs[3] += 1
            elif what == "backwards":
                rs[1], rs[2] = rs[2], rs[1]
            else:
                mr = max(rows) - 1
            table = table.to(DEV)
            cc = capi.masw_paged_cache(c.k, c.v, table, c.ks, c.vs)
            T = sum(rows)
            q = bf16(T, 4, 64, seed=2)
            o, lse = torch.zeros_like(q), torch.zeros(T, 4, device=DEV)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            capi.masw_paged_attn(cc, ints(kvl), q, o, lse, row_start=ints(rs), max_rows=mr, status=status)
            torch.cuda.synchronize()
            assert status.item() == capi.MASW_EINVAL, (rows, what)
            if what in ("page", "page_negative", "length"):       # the other sequences are served
                sub = [*range(rows[0]), T - 1]
                check_attention(c.mirror(), [c.table[0].tolist(), c.table[2].tolist()], [kv[0], kv[2]], [0, rows[0], rows[0] + 1],
                                q[sub], o[sub], lse[sub])


# ---------------------------------------------------------------- together --

@pytest.mark.parametrize("dtype,d", [("e4m3", 128), ("bf16", 128), ("e4m3", 64)])
def test_prompt_then_speculative_steps(dtype, d):
    """A prompt in two chunks, then verify blocks of which a part is rejected, as a server runs them: append, attend,
    accept greedily, shorten the lengths; against the oracle at every step."""
    hkv, hq, page, L = 2, 6, 16, 3
    cap = [200, 200]
    c = Cache(cap, hkv, d, page, dtype, seed=20)
    mirror = c.mirror()
    cs = tables(256, d)
    rope = capi.masw_rope(cs.to(DEV))
    table = c.table.tolist()
    kv = [0, 0]

    def step(n, seed):
        nonlocal kv
        kv = [a + b for a, b in zip(kv, n)]
        rs, T = starts(n), sum(n)
        q, k, v = bf16(T, hq, d, seed=seed), bf16(T, hkv, d, seed=seed + 1, mul=2.0 ** (seed % 5 - 2)), bf16(T, hkv, d, seed=seed + 2)
        qr, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(T, hq, device=DEV)
        capi.masw_paged_append(c.c, ints(kv), k, v, rope=rope, q=q, q_out=qr, row_start=ints(rs))
        capi.masw_paged_attn(c.c, ints(kv), qr, o, lse, row_start=ints(rs), max_rows=max(n))
        wq = po.append(mirror, table, kv, rs, np64(k), np64(v), cs.numpy(), False, None, np64(q))
        assert np.array_equal(np64(qr), wq)
        check_attention(mirror, table, kv, rs, qr, o, lse)
        return o

    step([60, 33], 1)
    step([41, 64], 4)
    for i in range(4):
        o = step([L + 1, L + 1], 10 * i + 7)
        logits = o.reshape(2, L + 1, hq * d)[:, :, :100].contiguous()
        tokens, n_emit = torch.empty(2, L + 1, dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
        draft = logits.argmax(-1)[:, :L].int().contiguous()
        draft[0, i % L] += 1                                     # a wrong draft: the rest of its block is rejected
        capi.masw_greedy_accept(logits, draft, tokens, n_emit)
        assert n_emit.tolist() == [i % L + 1, L + 1]
        kv = [a - (L + 1) + e for a, e in zip(kv, n_emit.tolist())]
    got = c.mirror()
    for b in range(2):
        for p in range(kv[b]):
            assert np.array_equal(got["k"][table[b][p // page], :, p % page], mirror["k"][table[b][p // page], :, p % page])


def test_captured_steps_replay_with_new_lengths():
    """append + attention captured once and replayed: lengths, rows and page table are read on the device."""
    hkv, hq, d, page = 2, 8, 128, 64
    for n0 in (2, 30):
        c = Cache([700, 700], hkv, d, page, "e4m3", seed=30)
        T = 2 * n0
        q, k, v = bf16(T, hq, d), bf16(T, hkv, d, seed=1), bf16(T, hkv, d, seed=2)
        qr, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(T, hq, device=DEV)
        kv, rs = ints([n0, n0]), ints([0, n0, T])
        cs = tables(1024, d)
        rope = capi.masw_rope(cs.to(DEV))
        ws = torch.empty(capi.masw_paged_workspace_bytes(c.c, T, T, hq), dtype=torch.uint8, device=DEV)
        ws.fill_(0xA5)

        def call():
            capi.masw_paged_append(c.c, kv, k, v, rope=rope, q=q, q_out=qr, row_start=rs)
            capi.masw_paged_attn(c.c, kv, qr, o, lse, row_start=rs, max_rows=T, workspace=ws)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            call()
        for lens, split in (([300, 40], n0), ([699, 257], 1), ([64, 128], T)):
            rows = [0, split, T]
            lens = [max(lens[0], split), max(lens[1], T - split)]
            kv.copy_(ints(lens))
            rs.copy_(ints(rows))
            q.copy_(bf16(T, hq, d, seed=lens[0]))
            want = c.mirror()
            graph.replay()
            torch.cuda.synchronize()
            wq = po.append(want, c.table.tolist(), lens, rows, np64(k), np64(v), cs.numpy(), False, None, np64(q))
            assert np.array_equal(np64(qr), wq) and np.array_equal(c.mirror()["k"], want["k"])
            check_attention(want, c.table.tolist(), lens, rows, qr, o, lse)


def test_two_streams_with_a_workspace_each_and_results_that_repeat():
    c = Cache([3000, 1500, 800], 2, 128, 64, "e4m3", seed=40)
    kv, n = [3000, 1500, 800], [1, 4, 2]
    q = bf16(7, 8, 128, seed=1)
    kvd, rs = ints(kv), ints(starts(n))
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(6):
        with torch.cuda.stream(streams[rep % 2]):
            o, lse = torch.empty_like(q), torch.empty(7, 8, device=DEV)
            capi.masw_paged_attn(c.c, kvd, q, o, lse, row_start=rs, max_rows=4)
            outs.append((o, lse))
    torch.cuda.synchronize()
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    check_attention(c.mirror(), c.table.tolist(), kv, starts(n), q, *outs[0])
