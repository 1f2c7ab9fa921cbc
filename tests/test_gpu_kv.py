"""The paged key/value cache on the GPU (append with rotation, read-back, attention)
against the fp64 oracle. Slots that no token occupies hold NaN and table entries that
no visible position needs hold an invalid page, so a read of either shows."""
import numpy as np
import pytest
import torch

from kv_cases import Cache, attention_reference
from oracle import paged
from transformer_layer_residual_b200 import fnl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle(cuda_device):
    h = fnl.Handle(0)
    yield h
    h.close()


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _cu(new):
    return _i32(np.concatenate([[0], np.cumsum(new)]))


def _dev(c, table=None):
    """(KVCache, table) of a CPU case on the GPU."""
    t = [None if x is None else x.cuda() for x in c.pages + c.scales]
    return fnl.KVCache(*t), (c.table if table is None else table).cuda()


def _check_attention(h, c, new, Hq, window=0, sinks=0, scale=None, tail=2, table=None, max_q=None, seed=0):
    """Runs a packed batch with `tail` rows behind its last sequence; checks outputs,
    lse, the rows behind, and that a second run gives the same bits."""
    M = sum(new) + tail
    g = torch.Generator().manual_seed(1000 + seed)
    q = torch.randn(Hq, M, c.D, generator=g).to(torch.bfloat16)
    scale = c.D ** -0.5 if scale is None else scale
    cache, tab = _dev(c, table)
    batch = fnl.KVBatch(_cu(new), _i32(c.lens), tab, max(new) if max_q is None else max_q)
    runs = []
    for _ in range(2):
        out = torch.full((M, Hq * c.D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, M), 7.0, device="cuda")
        fnl.paged_attention(h, cache, batch, q.cuda(), scale=scale, window=window, sinks=sinks, out=out, lse=lse)
        h.check()
        runs.append((out.cpu(), lse.cpu()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    ref, tol, rl, tl = attention_reference(c, new, q, scale, window, sinks)
    n = sum(new)
    got = runs[0][0].double().numpy().reshape(M, Hq, c.D)
    gl = runs[0][1].double().numpy()
    assert np.all(got[n:] == 7.0) and np.all(gl[:, n:] == 7.0)
    off = np.abs(got[:n] - ref[:n])
    assert np.all(off <= tol[:n]), f"out off by {np.max(off / np.maximum(tol[:n], 1e-30))} of its bound"
    none = np.isneginf(rl[:, :n])
    assert np.array_equal(none, np.isneginf(gl[:, :n]))
    assert np.all(got[:n][none.T] == 0)
    off = np.abs(np.where(none, 0, gl[:, :n]) - np.where(none, 0, rl[:, :n]))
    assert np.all(off <= tl[:, :n]), f"lse off by {np.max(off / tl[:, :n])} of its bound"
    return h.last_plan()


FMT = pytest.mark.parametrize("fmt", ["bf16", "int4"])


@FMT
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 2), (7, 1), (8, 1), (16, 1)])
def test_decode(handle, fmt, D, page, Hq, Hkv):
    """One new token each: lengths around the tiles, one token, no sequence length, no new token."""
    lens = [1, 2, 31, 32, 33, 0, 127, 128, 129, 255, 300, 513]
    new = [1] * len(lens)
    new[5] = 0
    new[9] = 0
    c = Cache(fmt, lens, Hkv, D, page, seed=D + Hq)
    assert "split" in _check_attention(handle, c, new, Hq)


@FMT
@pytest.mark.parametrize("D", [64, 128])
def test_decode_long_shared_by_blocks(handle, fmt, D):
    """Few long sequences: every head's keys are split over many blocks, unevenly."""
    c = Cache(fmt, [5001, 3, 2600], 2, D, 128, seed=5)
    _check_attention(handle, c, [1, 1, 1], 8)
    _check_attention(handle, c, [2, 1, 0], 8, seed=1)


@FMT
def test_decode_many_short(handle, fmt):
    """More sequences than threads of a block, some empty."""
    g = np.random.default_rng(8)
    lens = g.integers(1, 60, 700).tolist()
    new = [int(x) for x in g.integers(0, 2, 700)]
    c = Cache(fmt, lens, 2, 64, 16, seed=6)
    _check_attention(handle, c, new, 4, max_q=1)


@FMT
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (40, 0), (64, 4), (200, 33), (1000, 5), (33, 700)])
def test_decode_window(handle, fmt, window, sinks):
    """A window and sinks; pages that have left every window are invalid in the table."""
    lens = [1, 30, 64, 65, 200, 431, 640]
    c = Cache(fmt, lens, 2, 64, 16, seed=9)
    table = c.table.clone()
    for b, n in enumerate(lens):
        for i in range(table.shape[1]):
            if i * 16 >= sinks and (i + 1) * 16 <= n - window:
                table[b, i] = 1 << 30
    _check_attention(handle, c, [1] * len(lens), 8, window, sinks, table=table)


@FMT
def test_few_tokens_each(handle, fmt):
    """Several new tokens of a sequence in one piece, with a window between them."""
    c = Cache(fmt, [3, 4, 90, 260], 2, 128, 32, seed=10)
    for window, sinks in [(0, 0), (17, 0), (40, 6)]:
        _check_attention(handle, c, [3, 1, 4, 2], 8, window, sinks)


@FMT
@pytest.mark.parametrize("D,page,Hq,Hkv", [(64, 16, 4, 2), (128, 64, 6, 2), (128, 128, 7, 1), (64, 32, 2, 2),
                                            (128, 16, 16, 2), (128, 1024, 5, 1)])
def test_prompts(handle, fmt, D, page, Hq, Hkv):
    """Many new tokens: whole prompts, prompts continued, one token, none, lengths around the tiles."""
    new = [1, 64, 65, 0, 127, 200, 17, 128]
    lens = [1, 64, 65, 40, 255, 200, 300, 500]
    c = Cache(fmt, lens, Hkv, D, page, seed=D + page)
    _check_attention(handle, c, new, Hq)


@FMT
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 2), (64, 0), (100, 4), (130, 70), (300, 1)])
def test_prompts_window(handle, fmt, window, sinks):
    new, lens = [150, 3, 260, 70], [150, 260, 400, 70]
    c = Cache(fmt, lens, 2, 128, 32, seed=12)
    table = c.table.clone()
    for b, n in enumerate(lens):
        for i in range(table.shape[1]):
            if i * 32 >= sinks and (i + 1) * 32 <= n - new[b] + 1 - window:
                table[b, i] = -7
    _check_attention(handle, c, new, 6, window, sinks, table=table)


@FMT
@pytest.mark.parametrize("n", [1, 9, 40])
def test_large_scores_and_offsets(handle, fmt, n):
    """Scores of a few hundred (the maximum moves far) and values off zero."""
    c = Cache(fmt, [400, 77], 1, 64, 32, seed=13, spread=4.0)
    _check_attention(handle, c, [n, n], 4, scale=1.0)


@FMT
def test_sequence_shorter_than_its_new_tokens(handle, fmt):
    """kv_len < new tokens: reported by check(), nothing outside the buffers is touched."""
    c = Cache(fmt, [20, 2], 1, 64, 16, seed=14)
    cache, tab = _dev(c)
    q = torch.randn(2, 6, 64, device="cuda").to(torch.bfloat16)
    batch = fnl.KVBatch(_cu([1, 5]), _i32([20, 2]), tab, 5)
    fnl.paged_attention(handle, cache, batch, q)
    with pytest.raises(fnl.FnlError, match="status 9"):
        handle.check()
    _check_attention(handle, c, [2, 1], 2)   # the handle works on


@FMT
@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, False), (64, False), (128, False), (48, True), (128, True)])
@pytest.mark.parametrize("D,page,Hq,Hkv", [(64, 16, 4, 2), (128, 64, 14, 2), (128, 128, 3, 3)])
def test_append(handle, fmt, rot, interleaved, D, page, Hq, Hkv):
    """Pages, scales and rotated q bit for bit; untouched slots and rows keep their bits."""
    if rot > D:
        pytest.skip("rot_dim <= D")
    new, before = [1, 0, 40, 3, 130, 1], [0, 5, 30, 16, 1, 127]
    lens = [a + b for a, b in zip(new, before)]
    c = Cache(fmt, lens, Hkv, D, page, seed=rot + D)
    M, n = sum(new) + 3, sum(new)
    g = torch.Generator().manual_seed(rot)
    q = torch.randn(Hq, M, D, generator=g).to(torch.bfloat16)
    k = torch.randn(Hkv, M, D, generator=g).to(torch.bfloat16)
    v = torch.randn(Hkv, M, D, generator=g).to(torch.bfloat16)
    ang = torch.rand(max(lens), rot // 2, generator=g, dtype=torch.float64) * 400
    cos, sin = ang.cos().float(), ang.sin().float()
    pos = np.concatenate([np.arange(b, b + a) for a, b in zip(new, before)])
    cache, tab = _dev(c)
    batch = fnl.KVBatch(_cu(new), _i32(lens), tab, max(new))
    q_out = torch.full_like(q, 7.0).cuda()
    if rot:
        got = fnl.rope_append_kv(handle, cache, batch, q.cuda(), k.cuda(), v.cuda(), cos.cuda(), sin.cuda(),
                                 interleaved=interleaved, q_out=q_out)["q"]
        want = torch.full_like(q, 7.0)
        want[:, :n] = torch.from_numpy(paged.rotate(q[:, :n].double().numpy(), cos[pos].numpy(), sin[pos].numpy(),
                                                    interleaved)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)
        k = torch.from_numpy(paged.rotate(k[:, :n].double().numpy(), cos[pos].numpy(), sin[pos].numpy(),
                                          interleaved)).to(torch.bfloat16)
    else:
        qd = q.cuda()
        assert fnl.rope_append_kv(handle, cache, batch, qd, k.cuda(), v.cuda())["q"] is qd
    handle.check()
    at = 0
    for b, m in enumerate(new):   # the oracle's cache with the same rows stored
        ids = c.table[b].tolist()
        for i, x in enumerate((k, v)):
            c.store(i, ids, before[b], x[:, at:at + m])
        at += m
    for got, want in ((cache.k, c.pages[0]), (cache.v, c.pages[1]), (cache.k_scale, c.scales[0]),
                      (cache.v_scale, c.scales[1])):
        if want is not None:
            bits = torch.uint8 if want.dtype == torch.uint8 else torch.int16
            assert torch.equal(got.cpu().view(bits), want.view(bits))
    back = fnl.kv_gather(handle, cache, batch, k=torch.full((Hkv, M, D), 7.0, dtype=torch.bfloat16, device="cuda"))
    handle.check()
    for i, (name, x) in enumerate((("k", k), ("v", v))):
        x = x[:, :n].double().numpy()
        if fmt == "int4":
            x = paged.int4_values(*paged.int4_rows(x))
        assert torch.equal(back[name][:, :n].cpu(), torch.from_numpy(x).to(torch.bfloat16))
    assert torch.all(back["k"][:, n:] == 7.0)


def test_append_in_place_and_rows_that_are_constant_or_tiny(handle):
    """q_out = q; 4-bit rows whose values are equal, subnormal, or of one sign."""
    D, page = 64, 16
    k = torch.zeros(1, 6, D, dtype=torch.bfloat16)
    k[0, 0] = 3.0
    k[0, 1, 0] = 1e-39
    k[0, 2] = torch.linspace(100, 101, D).to(torch.bfloat16)
    k[0, 3] = -torch.linspace(0, 1e30, D).to(torch.bfloat16)
    k[0, 4, 5] = -2.0
    k[0, 5] = torch.arange(D).to(torch.bfloat16)
    v = -k
    cache = fnl.KVCache.empty(2, page, 1, D, "int4")
    batch = fnl.KVBatch(_cu([6]), _i32([6]), _i32([1]).view(1, 1), 6)
    q = torch.randn(2, 6, D).to(torch.bfloat16)
    cos, sin = torch.zeros(6, 32), torch.ones(6, 32)   # a quarter turn: (a, b) -> (-b, a)
    qd = q.cuda()
    assert fnl.rope_append_kv(handle, cache, batch, qd, k.cuda(), v.cuda(), cos.cuda(), sin.cuda(), q_out=qd)["q"] is qd
    handle.check()
    assert torch.equal(qd.cpu(), torch.cat([-q[..., 32:], q[..., :32]], -1))
    back = fnl.kv_gather(handle, cache, batch, M=6)
    kk = torch.cat([-k[..., 32:], k[..., :32]], -1)
    for name, x in (("k", kk), ("v", v)):
        want = paged.int4_values(*paged.int4_rows(x.double().numpy()))
        assert torch.equal(back[name].cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_bad_pages_and_positions_are_reported(handle):
    """A page outside the cache, a position outside the block table or the rotation
    table, a sequence over max_q: device code 9, the good rows stored, the rest left."""
    D, page = 64, 16
    k = torch.randn(1, 4, D).to(torch.bfloat16).cuda()
    for lens, tab, limit, max_q in (([4, 40], [[0, 0], [1, 99]], 64, 2), ([4, 40], [[0, 0], [1, 2]], 64, 2),
                                    ([4, 20], [[0, 0], [1, 2]], 19, 2), ([4, 20], [[0, 0], [1, 2]], 64, 1)):
        cache = fnl.KVCache(*(torch.full((3, 1, page, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        batch = fnl.KVBatch(_cu([2, 2]), _i32(lens), torch.tensor(tab, dtype=torch.int32, device="cuda"), max_q)
        one, zero = torch.ones(limit, 32, device="cuda"), torch.zeros(limit, 32, device="cuda")
        fnl.rope_append_kv(handle, cache, batch, k, k, k, one, zero)
        with pytest.raises(fnl.FnlError, match="status 9"):
            handle.check()
        if max_q == 2:
            assert torch.equal(cache.k[0, 0, 2:4], k[0, :2]) and torch.all(cache.k[0, 0, 4:] == 7.0)
            fnl.paged_attention(handle, cache, batch, k)
            if limit != 19:
                with pytest.raises(fnl.FnlError, match="status 9"):
                    handle.check()
    handle.check()


def test_strided_pages(handle):
    """k and v as the halves of one [num_pages, 2, ...] allocation."""
    D, page, Hkv = 64, 16, 2
    for fmt in ("bf16", "int4"):
        c = Cache(fmt, [50, 17], Hkv, D, page, seed=21)
        both = torch.stack(c.pages, 1).cuda()
        sc = [None, None]
        if fmt == "int4":
            scales = torch.stack(c.scales, 1).cuda()
            sc = [scales[:, 0], scales[:, 1]]
        cache = fnl.KVCache(both[:, 0], both[:, 1], *sc)
        batch = fnl.KVBatch(_cu([20, 1]), _i32(c.lens), c.table.cuda(), 20)
        q = torch.randn(4, 21, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
        got = fnl.paged_attention(handle, cache, batch, q.cuda())["out"]
        dense, tab = _dev(c)
        assert torch.equal(got, fnl.paged_attention(handle, dense, fnl.KVBatch(_cu([20, 1]), _i32(c.lens), tab, 20),
                                                    q.cuda())["out"])
        back = fnl.kv_gather(handle, cache, fnl.KVBatch(_cu([50, 17]), _i32(c.lens), c.table.cuda(), 50), M=67)
        handle.check()
        for i, n in enumerate(("k", "v")):
            want = np.concatenate([np.stack([c.parts(b, i, h)[0] for h in range(Hkv)]) for b in range(2)], 1)
            assert torch.equal(back[n].cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_far_pages(handle):
    """Offsets past 2^31 elements inside one cache."""
    D, page, Hkv = 128, 1024, 8
    n = (1 << 31) // (Hkv * page * D) + 3   # pages
    k = torch.empty(n, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    cache = fnl.KVCache(k, v)
    g = torch.Generator().manual_seed(3)
    q, x, y = (torch.randn(h, 3, D, generator=g).to(torch.bfloat16).cuda() for h in (16, Hkv, Hkv))
    outs = []
    for first in (0, n - 2):
        tab = torch.tensor([[first + 1, first]], dtype=torch.int32, device="cuda")
        k[first:first + 2] = torch.linspace(-1, 1, D, device="cuda").to(torch.bfloat16)
        v[first:first + 2] = torch.linspace(-1, 1, page, device="cuda").to(torch.bfloat16)[:, None]
        batch = fnl.KVBatch(_cu([3]), _i32([1100]), tab, 3)
        fnl.rope_append_kv(handle, cache, batch, q, x, y)
        assert torch.equal(k[first, :, 73:76], x) and torch.equal(v[first, :, 73:76], y)
        for max_q in (3, 64):
            outs.append(fnl.paged_attention(handle, cache, fnl.KVBatch(_cu([3]), _i32([1100]), tab, max_q), q)["out"])
    handle.check()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    del k, v, cache
    torch.cuda.empty_cache()


@FMT
def test_streams_and_a_replayed_graph(handle, fmt):
    """A decode step captured once and replayed over growing sequences, on a stream of
    its own; another handle works on another stream meanwhile."""
    Hq, Hkv, D, page, B = 8, 2, 64, 16, 3
    g = torch.Generator().manual_seed(31)
    steps = 20
    q, k, v = (torch.randn(steps, h, B, D, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    ang = torch.rand(200, D // 2, generator=g) * 6
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    tab = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    lens0 = [1, 30, 17]

    def caches():
        c = fnl.KVCache.empty(B * 4, page, Hkv, D, fmt)
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.zero_()
        return c

    def step(h, c, batch, qs, ks, vs, out):
        r = fnl.rope_append_kv(h, c, batch, qs, ks, vs, cos, sin)["q"]
        fnl.paged_attention(h, c, batch, r, out=out)

    # eager, on the current stream
    c0, kv = caches(), _i32(lens0)
    batch = fnl.KVBatch(_cu([1] * B), kv, tab, 1)
    eager = []
    for t in range(steps):
        out = torch.empty(B, Hq * D, dtype=torch.bfloat16, device="cuda")
        step(handle, c0, batch, q[t], k[t], v[t], out)
        eager.append(out)
        kv += 1
    # captured once, replayed; a second handle on another stream in between
    c1, kv1 = caches(), _i32(lens0)
    batch1 = fnl.KVBatch(_cu([1] * B), kv1, tab, 1)
    qs, ks, vs = (torch.empty_like(x[0]) for x in (q, k, v))
    out1 = torch.empty(B, Hq * D, dtype=torch.bfloat16, device="cuda")
    h2 = fnl.Handle(0)
    c2, kv2 = caches(), _i32(lens0)
    batch2 = fnl.KVBatch(_cu([1] * B), kv2, tab, 1)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(handle, c1, batch1, qs, ks, vs, out1)
    got, got2 = [], []
    for t in range(steps):
        with torch.cuda.stream(side):
            qs.copy_(q[t]); ks.copy_(k[t]); vs.copy_(v[t])
            graph.replay()
            got.append(out1.clone())
            kv1 += 1
        with torch.cuda.stream(other):
            o = torch.empty_like(out1)
            step(h2, c2, batch2, q[t], k[t], v[t], o)
            got2.append(o)
            kv2 += 1
    torch.cuda.synchronize()
    handle.check()
    h2.check()
    h2.close()
    for t in range(steps):
        assert torch.equal(eager[t], got[t]) and torch.equal(eager[t], got2[t]), t


@FMT
@pytest.mark.parametrize("rotary", [True, False])
def test_attention_half_of_a_layer(handle, fmt, rotary):
    """As a layer runs: the QKV op, the rotation and append, the attention, the output
    projection onto the residual stream; two prompts, then three decode steps. Each
    stage is held against the oracle on the stage's own inputs; the residual stream's
    dtype rounding is one half step, the projection's operands are bf16 products in
    fp32 (checked elsewhere), so the last stage compares with fp64 at 1e-2."""
    K, Hq, Hkv, D, page = 256, 4, 2, 64, 16
    g = torch.Generator().manual_seed(41)
    W = (torch.randn((Hq + 2 * Hkv) * D, K, generator=g) / K ** 0.5).to(torch.bfloat16)
    Wo = (torch.randn(K, Hq * D, generator=g) / (Hq * D) ** 0.5).to(torch.bfloat16)
    gamma = torch.ones(K, dtype=torch.bfloat16)
    ang = torch.outer(torch.arange(128, dtype=torch.float64), 10000.0 ** (-torch.arange(D // 2) / (D / 2)))
    cos, sin = (ang.cos().float().cuda(), ang.sin().float().cuda()) if rotary else (None, None)
    c = Cache(fmt, [0, 0], Hkv, D, page, seed=1, spare=12)
    cache, _ = _dev(c)
    table = torch.arange(12, dtype=torch.int32).view(2, 6)
    seen = [[np.zeros((Hkv, 0, D)) for _ in range(2)] for _ in range(2)]
    lens = [0, 0]
    for new in ([37, 50], [1, 1], [1, 1], [1, 1]):
        M = sum(new)
        lens = [a + b for a, b in zip(lens, new)]
        x, r = (torch.randn(M, K, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        batch = fnl.KVBatch(_cu(new), _i32(lens), table.cuda(), max(new))
        o = fnl.add_norm_qkv(handle, x, r, gamma.cuda(), None, W.cuda(), Hq, Hkv, D)
        q = fnl.rope_append_kv(handle, cache, batch, o["q"], o["k"], o["v"], cos, sin)["q"]
        a = fnl.paged_attention(handle, cache, batch, q)["out"]
        y = fnl.linear_add_residual(handle, a, Wo.cuda(), o["residual_out"])["out"]
        handle.check()
        at = 0
        c.lens, c.dense = list(lens), []
        k = o["k"].double().cpu().numpy()
        if rotary:
            pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
            k = paged.rotate(k, cos.cpu().numpy()[pos], sin.cpu().numpy()[pos])
        v = o["v"].double().cpu().numpy()
        for b, m in enumerate(new):
            for i, t in enumerate((k, v)):
                seen[b][i] = np.concatenate([seen[b][i], t[:, at:at + m]], 1)
            c.dense.append([torch.from_numpy(t) for t in seen[b]])
            at += m
        ref, tol, _, _ = attention_reference(c, new, q.cpu(), D ** -0.5)
        assert np.all(np.abs(a.double().cpu().numpy().reshape(M, Hq, D) - ref) <= tol)
        ref = o["residual_out"].double() + a.double() @ Wo.double().cuda().T
        assert torch.all((y.double() - ref).abs() <= 1e-2 + 1e-2 * ref.abs())


def test_refusals(handle):
    D, page = 64, 16
    cache = fnl.KVCache.empty(4, page, 2, D)
    tab = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    batch = fnl.KVBatch(_cu([2]), _i32([2]), tab, 2)
    q = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, D, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(8, D // 2, device="cuda")

    def refused(status, f, *a, **kw):
        with pytest.raises(fnl.FnlError) as e:
            f(handle, *a, **kw)
        assert e.value.status == status, e.value

    att, app, back = fnl.paged_attention, fnl.rope_append_kv, fnl.kv_gather
    refused(1, att, cache, batch, q, window=-1)
    refused(1, att, cache, batch, q, sinks=2)
    refused(1, att, cache, batch, q, scale=0.0)
    refused(1, att, cache, batch, q, scale=float("nan"))
    refused(1, att, cache, batch, q[:3])
    refused(1, att, cache, fnl.KVBatch(_cu([2]), _i32([2]), tab, 0), q)
    refused(1, att, cache, fnl.KVBatch(_cu([2]), _i32([2]), tab, -1), q)
    refused(3, att, cache, batch, q, out=q.view(2, 4 * D))
    refused(3, att, cache, batch, q, out=cache.k.view(-1)[:2 * 4 * D].view(2, 4 * D))
    refused(3, att, cache, batch, q, lse=t.view(-1)[:8].view(4, 2), out=t.view(torch.bfloat16).view(-1)[:512].view(2, 256))
    odd = torch.zeros(2 * 4 * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 4 * D)
    refused(2, att, cache, batch, q, out=odd)
    refused(1, app, cache, batch, q, k, k, t[:, :4].contiguous(), t[:, :4].contiguous())      # rot_dim 8
    refused(1, app, cache, batch, q[:1], k, k, t, t.clone())                                   # Hq < Hkv
    big = torch.zeros(4 * 2 * D + 64, dtype=torch.bfloat16, device="cuda")
    refused(3, app, cache, batch, big[:4 * 2 * D].view(4, 2, D), k, k, t, t.clone(), q_out=big[64:].view(4, 2, D))
    refused(3, app, cache, batch, q, cache.k.view(-1)[:256].view(2, 2, D), k)
    refused(3, back, cache, batch, k=k, v=k)
    for bad in (fnl.KVCache.empty(4, 24, 2, D), fnl.KVCache.empty(4, 8, 2, D), fnl.KVCache.empty(4, 2048, 2, D)):
        refused(4, att, bad, batch, q)
    refused(4, att, fnl.KVCache.empty(4, 16, 2, 96), batch, torch.zeros(4, 2, 96, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        app(handle, cache, batch, q, k, k, t)                       # cos without sin
    with pytest.raises(ValueError):
        app(handle, cache, batch, q, k, k, q_out=q)                 # q_out without a rotation
    with pytest.raises(ValueError):
        fnl.KVCache(cache.k, cache.v, cache.k, cache.v)             # scales of a bf16 cache
    with pytest.raises(ValueError):
        fnl.KVCache(cache.k.transpose(1, 2), cache.v.transpose(1, 2))
    with pytest.raises(ValueError):
        fnl.KVBatch(_cu([2]), _i32([2, 3]), tab, 2)
    # nothing to do: no rows, no sequences
    none = fnl.KVBatch(_i32([0]), _i32([]), tab[:0], 0)
    assert att(handle, cache, none, q[:, :0].contiguous())["out"].shape == (0, 4 * D)
    left = torch.full((2, 4 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.all(att(handle, cache, none, q, out=left)["out"] == 7.0)
    handle.check()


def test_a_wait_that_runs_out_is_reported(cuda_device):
    """Fault injection: the first block withholds its first key tile; the call ends, check()
    reports it, and the next call on the handle is right."""
    h = fnl.Handle(0, wait_ns=50_000_000, debug_stall_calls=1)
    c = Cache("bf16", [300, 200], 2, 128, 64, seed=50)
    cache, tab = _dev(c)
    batch = fnl.KVBatch(_cu([300, 200]), _i32(c.lens), tab, 300)
    q = torch.randn(4, 500, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    fnl.paged_attention(h, cache, batch, q)
    with pytest.raises(fnl.FnlError, match="status"):
        h.check()
    _check_attention(h, c, [300, 200], 4)
    h.close()


def test_prompts_of_many_sequences(handle):
    """More sequences than threads of a block, lengths of many kinds, some empty: the plan
    of the tensor-core form; then few tiles of long keys, shared by many blocks."""
    g = np.random.default_rng(60)
    new = [int(x) for x in g.integers(0, 9, 900)]
    lens = [n + int(x) for n, x in zip(new, g.integers(0, 40, 900))]
    lens = [max(n, 1) for n in lens]
    new[17], lens[17] = 300, 350
    c = Cache("bf16", lens, 1, 64, 16, seed=61)
    assert "tensor" in _check_attention(handle, c, new, 3)
    c = Cache("bf16", [6000, 50, 2900], 2, 128, 128, seed=62)
    _check_attention(handle, c, [20, 30, 0], 8)
    _check_attention(handle, c, [40, 1, 70], 8, window=1500, sinks=200)


def test_refusals_of_overlapping_pages(handle):
    """Pages that lie on one another: refused where they would be written, allowed where
    they are read (keys that are the values as well)."""
    Hkv, page, D = 2, 16, 64
    n = Hkv * page * D
    buf = torch.zeros(9 * n, dtype=torch.bfloat16, device="cuda")
    tab = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    batch = fnl.KVBatch(_cu([2]), _i32([2]), tab, 2)
    q = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(2, 2, D, dtype=torch.bfloat16, device="cuda")

    def pages(first, stride, count=4):
        return buf[first:].as_strided((count, Hkv, page, D), (stride, page * D, D, 1))

    with pytest.raises(ValueError, match="overlap"):
        fnl.KVCache(buf[:n].view(1, Hkv, page, D).expand(4, -1, -1, -1), pages(0, n))
    with pytest.raises(ValueError, match="overlap"):
        fnl.KVCache(pages(0, n - 16), pages(0, n - 16))
    for a, b in ((pages(0, n), pages(0, n)), (pages(0, n), pages(3 * n + n // 2, n)), (pages(3 * n + 16, n), pages(0, n)),
                 (pages(0, 2 * n), pages(n - 8, 2 * n)), (pages(n + 8, 2 * n), pages(0, 2 * n))):
        with pytest.raises(fnl.FnlError) as e:
            fnl.rope_append_kv(handle, fnl.KVCache(a, b), batch, None, k, k)
        assert e.value.status == 3, e.value
    for a, b in ((pages(0, n), pages(4 * n, n)), (pages(0, 2 * n), pages(n, 2 * n)), (pages(n, 2 * n), pages(0, 2 * n))):
        fnl.rope_append_kv(handle, fnl.KVCache(a, b), batch, None, k, k)
    same = fnl.KVCache(pages(0, n), pages(0, n))
    pages(0, n)[:] = 3.0
    assert torch.all(fnl.paged_attention(handle, same, batch, q)["out"] == 3.0)
    c = fnl.KVCache.empty(4, page, Hkv, D, "int4")
    with pytest.raises(fnl.FnlError) as e:
        fnl.rope_append_kv(handle, fnl.KVCache(c.k, c.v, c.k_scale, c.k_scale), batch, None, k, k)
    assert e.value.status == 3, e.value
    # more positions than the key tiles' counts hold
    far = fnl.KVBatch(_cu([2]), _i32([2]), torch.zeros(1, (1 << 26) + 1, dtype=torch.int32, device="cuda"), 2)
    with pytest.raises(fnl.FnlError) as e:
        fnl.paged_attention(handle, same, far, q)
    assert e.value.status == 4, e.value
    handle.check()


@FMT
def test_prompts_in_a_replayed_graph(cuda_device, fmt):
    """The tensor-core form captured as a handle's first call, replayed on other lengths
    (an empty sequence, no sequence longer than a row tile, one of every block's) and
    between eager calls of the split form on the same handle and stream."""
    Hq, Hkv, D, page, B, M = 8, 2, 64, 16, 3, 700
    c = Cache(fmt, [900, 700, 400], Hkv, D, page, seed=70)
    cache, tab = _dev(c)
    h, h0 = fnl.Handle(0), fnl.Handle(0)
    q = torch.randn(Hq, M, D, generator=torch.Generator().manual_seed(71)).to(torch.bfloat16).cuda()
    cu, kv = _cu([300, 200, 200]), _i32(c.lens)
    batch = fnl.KVBatch(cu, kv, tab, 500)
    out = torch.empty(M, Hq * D, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fnl.paged_attention(h, cache, batch, q, out=out, window=300, sinks=3)
    one = fnl.KVBatch(_cu([1, 1, 1]), _i32(c.lens), tab, 1)
    for new, lens in (([300, 200, 200], [900, 700, 400]), ([500, 0, 7], [600, 700, 7]), ([1, 1, 1], [1, 650, 399]),
                      ([0, 0, 0], [5, 5, 5])):
        want = torch.full_like(out, 7.0)
        fnl.paged_attention(h0, cache, fnl.KVBatch(_cu(new), _i32(lens), tab, 500), q, out=want, window=300, sinks=3)
        first = fnl.paged_attention(h0, cache, one, q[:, :3].contiguous())["out"]
        cu.copy_(_cu(new))
        kv.copy_(_i32(lens))
        out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
            got = fnl.paged_attention(h, cache, one, q[:, :3].contiguous())["out"]
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(got, first), new
    h.check()
    h0.check()
    h.close()
    h0.close()


@FMT
@pytest.mark.parametrize("n", [1, 40])
def test_sequences_that_share_pages(handle, fmt, n):
    """A common prefix kept once: the same bits as from copies of its pages."""
    Hq, Hkv, D, page = 8, 2, 64, 32
    c = Cache(fmt, [256 + n, 256 + n], Hkv, D, page, seed=80)
    cache, tab = _dev(c)
    q = torch.randn(Hq, 2 * n, D, generator=torch.Generator().manual_seed(81)).to(torch.bfloat16).cuda()
    shared = tab.clone()
    shared[1, :8] = tab[0, :8]
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t[tab[1, :8].long()] = t[tab[0, :8].long()]
    outs = [fnl.paged_attention(handle, cache, fnl.KVBatch(_cu([n, n]), _i32(c.lens), x, n), q)["out"] for x in (tab, shared)]
    handle.check()
    assert torch.equal(*outs)


def test_a_wait_that_runs_out_over_4_bit_pages(cuda_device):
    """The same for prompts over 4-bit pages, whose copies go through a ring of their own."""
    h = fnl.Handle(0, wait_ns=50_000_000, debug_stall_calls=1)
    c = Cache("int4", [300, 200], 2, 128, 64, seed=90)
    cache, tab = _dev(c)
    batch = fnl.KVBatch(_cu([300, 200]), _i32(c.lens), tab, 300)
    q = torch.randn(4, 500, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    fnl.paged_attention(h, cache, batch, q)
    with pytest.raises(fnl.FnlError, match="status"):
        h.check()
    _check_attention(h, c, [300, 200], 4)
    h.close()


@FMT
@pytest.mark.parametrize("B,n,ctx", [(1, 40, 5000), (6, 33, 700), (80, 70, 90), (100, 65, 10)])
def test_prompts_shared_or_whole(handle, fmt, B, n, ctx):
    """One long key axis over every block; few tiles taken whole; between one and two
    waves, and more tiles than the shared list holds."""
    g = np.random.default_rng(95 + B)
    new = [int(x) for x in g.integers(n // 2, n + 1, B)]
    c = Cache(fmt, [x + int(y) for x, y in zip(new, g.integers(ctx // 2, ctx + 1, B))], 2, 64, 64, seed=96)
    assert "tensor" in _check_attention(handle, c, new, 16 if B == 100 else 8)
