"""The paged-cache oracle pinned against torch's own types and closed forms (CPU)."""
import numpy as np
import torch

import oracle.paged_oracle as po


def test_e4m3_rounding_is_the_types():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    fin = every[np.isfinite(every)]
    assert np.array_equal(po.e4m3_round(fin), fin)
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=g) * s for s in (1e-3, 0.02, 1.0, 100.0)]).clamp(-448, 448)
    grid = np.unique(fin)
    x = torch.cat([x, torch.from_numpy((grid[1:] + grid[:-1]) / 2).float()])     # every tie
    assert np.array_equal(po.e4m3_round(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_bf16_rounding_is_the_types():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(20000, generator=g) * 7
    assert np.array_equal(po.bf16_round(x.double().numpy()), x.to(torch.bfloat16).double().numpy())


def test_scale_borders():
    for e in (-30, -9, 0, 5):
        assert po.pow2_scale(448.0 * 2.0 ** e) == 2.0 ** e
        assert po.pow2_scale(np.nextafter(448.0 * 2.0 ** e, np.inf)) == 2.0 ** (e + 1)
    assert po.pow2_scale(0.0) == 1.0 and po.pow2_scale(1e-40) == 2.0 ** -64


def test_rotation_turns_by_the_angle():
    g = np.random.default_rng(3)
    x, ang = g.standard_normal((2, 32)).astype(np.float32), g.uniform(-3, 3, 8)
    cs = np.concatenate([np.cos(ang), np.sin(ang)])
    for inter in (False, True):
        y = po.rotate(x, cs, inter)
        for i in range(8):
            a, b = (2 * i, 2 * i + 1) if inter else (i, 8 + i)
            z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * ang[i])
            assert np.allclose(y[:, a], z.real, atol=1e-6) and np.allclose(y[:, b], z.imag, atol=1e-6)
        assert np.array_equal(y[:, 16:], x[:, 16:].astype(np.float64))


def test_attention_equals_softmax_over_the_visible_keys():
    g = np.random.default_rng(4)
    P, hkv, D, kv, n = 16, 2, 64, 37, 3
    cache = {"k": g.standard_normal((4, hkv, P, D)), "v": g.standard_normal((4, hkv, P, D)), "k_scale": None, "v_scale": None}
    table, q = [[3, 0, 2, 1]], g.standard_normal((n, 4, D))
    o, lse, *_ = po.attention(cache, table, [kv], [0, n], q, window=9)
    K = np.concatenate([cache["k"][i] for i in table[0]], 1)[:, :kv]
    V = np.concatenate([cache["v"][i] for i in table[0]], 1)[:, :kv]
    for j in range(n):
        at = kv - n + j
        for h in range(4):
            x = torch.from_numpy(K[h // 2, at - 8:at + 1] @ q[j, h] / 8.0)
            assert np.allclose(o[j, h], (torch.softmax(x, 0).numpy()[:, None] * V[h // 2, at - 8:at + 1]).sum(0))
            assert np.isclose(lse[j, h], torch.logsumexp(x, 0).item())
    o, lse, *_ = po.attention(cache, table, [1], [0, 3], q)      # rows 0 and 1 stand before the first key
    assert not o[:2].any() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2]).all()
