"""Pins of the paged-cache oracle and the checks of the binding that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from kv_cases import Cache, attention_reference
from oracle import paged
from transformer_layer_residual_b200 import fnl


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64])
def test_rotation_is_a_complex_product(rot, interleaved):
    g = np.random.default_rng(rot)
    x = torch.randn(3, 5, 64, generator=torch.Generator().manual_seed(rot)).to(torch.bfloat16).double().numpy()
    ang = g.uniform(-50, 50, (5, rot // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    y = paged.rotate(x, cos, sin, interleaved)
    i = np.arange(rot // 2)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = (x[..., one] + 1j * x[..., two]) * (cos.astype(np.float64) + 1j * sin)
    # one bf16 rounding (2^-8 relative) and three fp32 ones of terms up to |x|
    mag = np.abs(x[..., one]) + np.abs(x[..., two])
    for got, ref in ((y[..., one], z.real), (y[..., two], z.imag)):
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -24 * mag * (1 + 2.0 ** -8))
    assert np.array_equal(y[..., rot:], x[..., rot:])
    # relative positions: the product of two rotated vectors depends on the angle difference only
    assert np.allclose(paged.rotate(x, np.ones_like(cos), np.zeros_like(sin), interleaved), x)


def test_int4_rows():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(200, 64, generator=g).to(torch.bfloat16).double().numpy() * 2.0 ** np.arange(-100, 100)[:, None]
    x[7] = 0.25            # a constant row
    x[8] = np.arange(64) % 16 + 5.0    # a row that the grid holds exactly
    c, s, lo = paged.int4_rows(x)
    y = paged.int4_values(c, s, lo)
    assert c.min() == 0 and c.max() == 15
    # half a step, and the fp32 rounding of the quotient (at most 15 wide) before it is rounded
    assert np.all(np.abs(y - x) <= s[:, None] * (0.5 + 16 * 2.0 ** -23))
    assert np.array_equal(y[7], x[7]) and s[7] == 0
    assert np.array_equal(y[8], x[8]) and s[8] == 1
    t = (x.max(-1) - x.min(-1)) / 15
    assert np.all(s >= t * (1 - 2.0 ** -23)) and np.all(s <= t * (1 + 2.0 ** -7))   # rounded up, by less than a step
    assert np.array_equal(lo, x.min(-1))
    packed = paged.pack_codes(c)
    assert np.array_equal(packed & 15, c[:, 0::2]) and np.array_equal(packed >> 4, c[:, 1::2])


def test_attention_loops():
    """Against per-element loops, with a window, sinks, and a token that sees nothing."""
    g = np.random.default_rng(3)
    q, k, v = g.normal(size=(4, 8)), g.normal(size=(6, 8)), g.normal(size=(6, 8))
    pos, window, sinks = [-1, 2, 4, 5], 2, 1
    out, lse, p = paged.attention(q, k, v, pos, 0.3, window, sinks)
    for i in range(4):
        seen = [j for j in range(6) if j <= pos[i] and (j > pos[i] - window or j < sinks)]
        w = [np.exp(0.3 * sum(q[i][d] * k[j][d] for d in range(8))) for j in seen]
        ref = sum(w[a] * v[j] for a, j in enumerate(seen)) / sum(w) if seen else np.zeros(8)
        assert np.allclose(out[i], ref, rtol=1e-12, atol=1e-14)
        assert (lse[i] == -np.inf) if not seen else abs(lse[i] - np.log(sum(w))) < 1e-12
        assert [j for j in range(6) if p[i][j] > 0] == seen


def test_reference_places_tokens():
    """Values that name their position: a one-hot softmax returns the token's own row."""
    c = Cache("bf16", [5, 0, 17], 2, 64, 16, seed=4)
    for b, n in enumerate(c.lens):
        for i in range(2):
            c.dense[b][i] = torch.zeros(2, n, 64, dtype=torch.bfloat16)
        for t in range(n):
            c.dense[b][0][:, t, t] = 1.0
            c.dense[b][1][:, t, 0] = t
    q = torch.zeros(4, 5, 64, dtype=torch.bfloat16)
    for m, t in enumerate([3, 4, 14, 15, 16]):
        q[:, m, t] = 2048.0
    out, _, _, _ = attention_reference(c, [2, 0, 3], q, 1.0)
    assert np.array_equal(out[:, 0, 0], [3, 4, 14, 15, 16])


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fnl.KVCache(k, k.clone())
    with pytest.raises(ValueError, match="bfloat16 or torch.uint8"):
        fnl.KVCache(k.float(), k.float())
    with pytest.raises(ValueError, match="num_pages"):
        fnl.KVCache(k[0], k[0])
    with pytest.raises(ValueError, match="format"):
        fnl.KVCache.empty(1, 16, 1, 64, format="fp4", device="cpu")
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fnl.KVBatch(i, i[:2], i.view(3, 1)[:2], 1)


def test_null_handle_is_refused():
    L = fnl.lib()
    c, b = ctypes.byref(fnl._KvCache()), ctypes.byref(fnl._KvBatch())
    assert L.fnl_rope_append_kv(None, None, c, b, 1, 1, None, None, None, None, None, 0, 0, 0, None) == 1
    assert L.fnl_kv_gather(None, None, c, b, 1, None, None) == 1
    assert L.fnl_paged_attention(None, None, c, b, 1, 1, None, ctypes.c_float(1), 0, 0, None, None) == 1
