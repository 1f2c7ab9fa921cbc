"""The paged key/value cache at the edges of what its entry points allow: NaN in q, sequences
without new tokens; a handle's options, and what it says of its calls."""
import gc

import numpy as np
import pytest
import torch

from kv_cases import Cache
from test_gpu_kv import _check_attention
from transformer_layer_residual_b200 import fnl

pytestmark = pytest.mark.gpu

FMT = pytest.mark.parametrize("fmt", ["bf16", "int4"])


@pytest.fixture(scope="module")
def handle(cuda_device):
    h = fnl.Handle(0)
    yield h
    h.close()


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _cu(new):
    return _i32(np.concatenate([[0], np.cumsum(new)]))


def _dev(c):
    """(KVCache, table) of a CPU case on the GPU."""
    return fnl.KVCache(*[None if x is None else x.cuda() for x in c.pages + c.scales]), c.table.cuda()


@FMT
@pytest.mark.parametrize("new,lens", [([1, 1], [70, 3000]), ([3, 2], [40, 3000]), ([40, 20], [60, 3000])])
def test_nan_in_q_stays_in_its_row(handle, fmt, new, lens):
    """A NaN in one head of one token gives NaN in that row's output and log-sum-exp, in
    every form and where a head's keys are shared by blocks; all other rows keep their bits."""
    Hq, Hkv, D = 8, 2, 64
    c = Cache(fmt, lens, Hkv, D, 32, seed=3)
    cache, tab = _dev(c)
    M = sum(new)
    batch = fnl.KVBatch(_cu(new), _i32(lens), tab, max(new))
    q = torch.randn(Hq, M, D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    bad = q.clone()
    rows = [(1, 0), (6, M - 1), (3, new[0])]   # (head, token): of the first sequence, of the long one
    for hq, m in rows:
        bad[hq, m, 5] = float("nan")
    got = []
    for x in (q, bad):
        lse = torch.full((Hq, M), 7.0, device="cuda")
        out = fnl.paged_attention(handle, cache, batch, x, lse=lse)["out"]
        got.append((out.view(M, Hq, D).cpu(), lse.cpu()))
    handle.check()
    hit = torch.zeros(M, Hq, dtype=torch.bool)
    for hq, m in rows:
        hit[m, hq] = True
    assert torch.isfinite(got[0][0].float()).all() and torch.isfinite(got[0][1]).all()
    assert torch.isnan(got[1][0][hit].float()).all() and torch.isnan(got[1][1].t()[hit]).all()
    assert torch.equal(got[1][0][~hit], got[0][0][~hit]) and torch.equal(got[1][1].t()[~hit], got[0][1].t()[~hit])


@FMT
@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("idle", [-1, 0, 1 << 30])
def test_length_of_a_sequence_without_new_tokens_is_not_used(handle, fmt, n, idle):
    """The free slots of a padded batch: whatever their kv_len, every call takes them alike."""
    Hq, Hkv, D = 4, 2, 64
    c = Cache(fmt, [50, 33], Hkv, D, 16, seed=5)
    cache, tab = _dev(c)
    table = torch.full((4, tab.shape[1]), -1, dtype=torch.int32, device="cuda")
    table[0], table[2] = tab
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(h, 2 * n, D, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    got = []
    for new, lens, t in (([n, n], [50, 33], tab), ([n, 0, n, 0], [50, idle, 33, idle], table)):
        batch = fnl.KVBatch(_cu(new), _i32(lens), t, n)
        fnl.rope_append_kv(handle, cache, batch, None, k, v)
        out = fnl.paged_attention(handle, cache, batch, q)["out"]
        back = fnl.kv_gather(handle, cache, batch, M=2 * n)
        handle.check()
        got.append((out, back["k"], back["v"]))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_last_plan_names_the_last_call(handle):
    c = fnl.KVCache.empty(4, 16, 2, 64)
    batch = fnl.KVBatch(_cu([3]), _i32([3]), _i32([2]).view(1, 1), 3)
    q, k = (torch.randn(h, 3, 64, device="cuda").to(torch.bfloat16) for h in (4, 2))
    fnl.rope_append_kv(handle, c, batch, None, k, k)
    assert handle.last_plan() == "paged append, grid 3"
    fnl.paged_attention(handle, c, batch, q)
    assert "paged attention" in handle.last_plan()
    fnl.kv_gather(handle, c, batch, M=3)
    assert handle.last_plan() == "paged read-back, grid 3"
    x, W = (torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda") for n in (3, 64))
    fnl.linear_add_residual(handle, x, W, x)
    assert "paged" not in handle.last_plan() and handle.last_plan()
    fnl.rope_append_kv(handle, c, batch, None, k, k)
    assert handle.last_plan() == "paged append, grid 3"
    handle.check()


@FMT
@pytest.mark.parametrize("ctas", [1, 3, 7])
def test_capped_grids(cuda_device, fmt, ctas):
    """max_ctas: long keys in few parts, many sequences and heads a block, more tiles than a block has threads."""
    h = fnl.Handle(0, max_ctas=ctas)
    c = Cache(fmt, [1500, 3, 700, 64], 2, 64, 32, seed=7)
    for new, Hq, form in (([1, 1, 0, 1], 8, "8 rows"), ([3, 1, 2, 1], 8, "16 rows"), ([40, 3, 300, 0], 4, "tensor-core")):
        plan = _check_attention(h, c, new, Hq, window=600, sinks=5)
        assert form in plan and plan.endswith(f"grid {ctas}"), plan
    c = Cache(fmt, [12] * 450, 1, 64, 16, seed=8)
    assert _check_attention(h, c, [9] * 450, 2).endswith(f"grid {ctas}")
    h.close()


@pytest.mark.parametrize("new", [[1, 1], [2, 1]])
@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out_in_the_split_form(cuda_device, D, new):
    """Fault injection in a decode call over 4-bit pages: the block that withholds its first
    copies ends, check() reports it, the next call on the handle is right. Calls without a
    bounded wait leave the injection armed."""
    h = fnl.Handle(0, wait_ns=50_000_000, debug_stall_calls=1)
    wide = Cache("bf16", [300, 200], 1, D, 64, seed=50)
    _check_attention(h, wide, new, 8)
    c = Cache("int4", [3000, 200], 1, D, 64, seed=51)
    cache, tab = _dev(c)
    batch = fnl.KVBatch(_cu(new), _i32(c.lens), tab, max(new))
    q = torch.randn(8, sum(new), D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    fnl.kv_gather(h, cache, batch, M=sum(new))
    fnl.paged_attention(h, cache, batch, q)
    assert "split" in h.last_plan()
    with pytest.raises(fnl.FnlError, match="status 1 "):
        h.check()
    _check_attention(h, c, new, 8)
    h.close()


def test_a_handle_without_paged_calls_holds_no_cache_workspace(cuda_device):
    """The workspace (39 MB on 148 SMs) comes with the first paged call, once, whether that
    is eager or captured; a handle that makes none neither holds nor checks it."""
    c = fnl.KVCache.empty(4, 16, 2, 64)
    batch = fnl.KVBatch(_cu([3]), _i32([3]), _i32([2]).view(1, 1), 3)
    q, k = (torch.randn(h, 3, 64, device="cuda").to(torch.bfloat16) for h in (4, 2))
    out = torch.empty(3, 4 * 64, dtype=torch.bfloat16, device="cuda")

    def calls(h):
        fnl.rope_append_kv(h, c, batch, None, k, k)
        fnl.paged_attention(h, c, batch, q, out=out)

    h = fnl.Handle(0)
    calls(h)           # (loads the kernels)
    h.check()
    h.close()
    want = out.clone()
    for captured in (False, True):
        out.fill_(7.0)
        torch.cuda.synchronize()
        gc.collect()
        torch.cuda.empty_cache()   # (as the start of a capture does)
        free = [torch.cuda.mem_get_info()[0]]
        h = fnl.Handle(0)
        h.check()
        free.append(torch.cuda.mem_get_info()[0])
        if captured:
            side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                calls(h)
            graph.replay()
        else:
            calls(h)
        h.check()
        free.append(torch.cuda.mem_get_info()[0])
        calls(h)
        h.check()
        free.append(torch.cuda.mem_get_info()[0])
        assert torch.equal(out, want)
        h.close()
        assert free[0] - free[1] < 8 << 20, free
        assert free[1] - free[2] > 16 << 20 and free[2] == free[3], free


@FMT
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("window,sinks", [(40, 4), (700, 500), (40, 500), (700, 4)])
def test_from_the_sinks_to_a_far_window(handle, fmt, D, page, window, sinks):
    """The keys between the sinks and the window take up whole tiles in every form (of 8 rows, of
    16, of prompts), and the table has no page there."""
    lens = [5001, 1, 3000]
    c = Cache(fmt, lens, 2, D, page, seed=window + sinks)
    for new, Hq, form in (([1, 1, 1], 16, "8 rows"), ([2, 1, 2], 16, "16 rows"), ([3, 0, 4], 4, "8 rows"), ([40, 1, 70], 6, "tensor")):
        table = c.table.clone()
        for b, n in enumerate(lens):
            for i in range(table.shape[1]):
                if i * page >= sinks and (i + 1) * page <= n - new[b] + 1 - window:
                    table[b, i] = 1 << 30
        assert form in _check_attention(handle, c, new, Hq, window, sinks, table=table)


@FMT
@pytest.mark.parametrize("D", [64, 128])
def test_long_heads_of_16_rows_over_many_blocks(handle, fmt, D):
    """Two key heads over every block: dozens of parts of 16 rows added, and one of a few."""
    c = Cache(fmt, [40001, 700], 1, D, 128, seed=100 + D)
    for new, Hq in (([1, 1], 16), ([2, 1], 8), ([2, 0], 7)):
        assert "16 rows" in _check_attention(handle, c, new, Hq)
