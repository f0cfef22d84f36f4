"""Workspaces of the bf16 calls on streams of the caller's."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BUSY = 200_000_000  # clock cycles, about 0.1 s: what is queued behind them has not run when the test goes on


@pytest.fixture(scope="module")
def daa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import decode_attention_append_gb300 as m
    m.device_error(reset=True)
    return m


@pytest.fixture(scope="module")
def batch(daa):
    """A decode batch whose keys are cut, so that its workspace is large: table, pool, new K, new V, q."""
    rng = np.random.default_rng(1)
    n, pages, hq, hkv, d = 64, 400, 32, 8, 128
    table = daa.PageTable.from_host(np.arange(n + 1), pages * np.arange(n + 1),
                                    rng.permutation(n * pages).astype(np.int32), np.full(n, 5), DEV)
    gen = torch.Generator(DEV).manual_seed(1)
    pool, k, v, q = (torch.randn(s, generator=gen, device=DEV, dtype=torch.bfloat16)
                     for s in ((n * pages, 2, hkv, 16, d), (n, hkv, d), (n, hkv, d), (n, hq, d)))
    return table, pool, k, v, q


def _calls(attn, b, planned):
    _, _, k, v, q = b
    if planned:
        attn.plan()
    return {"run": lambda out, s: attn.run(q, out=out, stream=s), "step": lambda out, s: attn.step(k, v, q, out=out, stream=s)}


@pytest.mark.parametrize("call", ["run", "step"])
@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("raw", [False, True])
def test_workspace_outlives_its_object(daa, batch, call, planned, raw):
    """An object dropped while a call is under way: its workspace is nobody else's until that has ended."""
    table, pool, _, _, q = batch
    attn = daa.BatchAttention(table, q.shape[1], pool)
    want = torch.empty_like(q)
    _calls(attn, batch, planned)[call](want, None)
    n = attn.workspace.numel()
    assert n > 1 << 20  # a block of its own
    del attn
    s, out = torch.cuda.Stream(), torch.empty_like(q)
    attn = daa.BatchAttention(table, q.shape[1], pool)
    at = attn.workspace.data_ptr()
    run = _calls(attn, batch, planned)[call]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    run(out, s.cuda_stream if raw else s)
    pending = not s.query()
    del attn, run
    other = torch.empty(n, dtype=torch.uint8, device=DEV)  # never written
    # not this memory, or on a stream that waits for the call
    safe = other.data_ptr() != at or not torch.cuda.current_stream().query()
    s.synchronize()
    assert pending and safe
    assert torch.equal(out, want) and daa.device_error(reset=True) == 0


@pytest.mark.parametrize("call", ["attention", "append", "tree", "run", "noalloc"])
def test_what_a_call_allocates_is_its_streams(daa, batch, call):
    """Output and workspace that a call makes are the named stream's memory: given back when the call returns, they are
    nobody else's before the stream has come to it."""
    table, pool, k, v, q = batch
    host = (table.h_qo_indptr, table.h_kv_indptr, table.h_last_page_len)
    dev = (table.qo_indptr, table.kv_indptr, table.page_indices, table.last_page_len)
    attn = daa.BatchAttention(table, q.shape[1], pool)
    need = attn.workspace.numel()
    if call == "run":
        attn.plan()
    mask = torch.ones(q.shape[0], 1, dtype=torch.int32, device=DEV)
    calls = {"attention": lambda s: daa.batch_attention(q, pool, *dev, host_indptr=host, stream=s),
             "append": lambda s: daa.append_attention(k, v, q, pool, *dev, host_indptr=host, stream=s),
             "tree": lambda s: daa.batch_attention_tree(q, pool, *dev, mask, host_indptr=host, stream=s),
             "run": lambda s: attn.run(q, stream=s),
             "noalloc": lambda s: daa.batch_attention_noalloc(q, pool, *dev, host, stream=s)}
    want = calls[call](None)
    torch.cuda.synchronize()
    for raw in (False, True):
        s = torch.cuda.Stream()
        held = lambda: sum(x["total_size"] for x in torch.cuda.memory_snapshot() if x["stream"] == s.cuda_stream)  # noqa: E731
        torch.cuda.empty_cache()
        before = held()
        out = calls[call](s.cuda_stream if raw else s)
        made = held() - before
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert made >= out.numel() * 2 + (need if call in ("attention", "append", "tree") else 0)
    assert daa.device_error(reset=True) == 0


@pytest.mark.parametrize("call", ["attention", "append", "tree"])
@pytest.mark.parametrize("raw", [False, True])
def test_lengths_are_read_on_the_stream_of_the_call(daa, batch, call, raw):
    """Without host copies a call reads the table from the device: behind what its stream holds."""
    table, pool, k, v, q = batch
    src = (table.qo_indptr, table.kv_indptr, table.page_indices, table.last_page_len)
    mask = torch.ones(q.shape[0], 1, dtype=torch.int32, device=DEV)
    calls = {"attention": daa.batch_attention, "append": lambda *a, **kw: daa.append_attention(k, v, *a, **kw),
             "tree": lambda *a, **kw: daa.batch_attention_tree(*a, mask, **kw)}
    want = calls[call](q, pool, *src)
    dst, s = [torch.zeros_like(x) for x in src], torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
        for d, x in zip(dst, src):
            d.copy_(x)
    out = calls[call](q, pool, *dst, stream=s.cuda_stream if raw else s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and daa.device_error(reset=True) == 0


def test_streams_of_other_libraries(daa, batch):
    """An object with a cuda_stream handle is a stream, as an integer is."""
    table, pool, k, v, q = batch
    host = (table.h_qo_indptr, table.h_kv_indptr, table.h_last_page_len)
    dev = (table.qo_indptr, table.kv_indptr, table.page_indices, table.last_page_len)
    s = torch.cuda.Stream()

    class Stream:
        cuda_stream = s.cuda_stream
    want = daa.batch_attention(q, pool, *dev, host_indptr=host)
    attn, copy = daa.BatchAttention(table, q.shape[1], pool), pool.clone()
    torch.cuda.synchronize()
    outs = [daa.batch_attention(q, pool, *dev, stream=Stream()),
            daa.append_attention(k, v, q, copy, *dev, host_indptr=host, stream=Stream()), attn.run(q, stream=Stream())]
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[2], want) and daa.device_error(reset=True) == 0


def test_object_dropped_during_a_capture(daa, batch):
    """An object that ran on the caller's stream, dropped while its own stream is being captured: the capture goes on, and the
    memory is kept for later."""
    table, pool, _, _, q = batch
    home, s = torch.cuda.Stream(), torch.cuda.Stream()
    want = daa.BatchAttention(table, q.shape[1], pool).run(q)
    x = torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        attn = daa.BatchAttention(table, q.shape[1], pool)
    out = attn.run(q, stream=s.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=home):
        x.add_(1)
        del attn
        x.add_(1)
    assert len(daa._late) == 1
    with torch.cuda.stream(home):
        other = daa.BatchAttention(table, q.shape[1], pool)
    again = other.run(q, stream=s.cuda_stream)
    del other
    assert not daa._late
    graph.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [2.0] * 4
    assert torch.equal(out, want) and torch.equal(again, want) and daa.device_error(reset=True) == 0


@pytest.mark.parametrize("raw", [False, True])
def test_first_call_on_a_stream_beside_a_capture(daa, batch, raw):
    """A call on a stream of its own while the constructor's stream is being captured stays out of the capture."""
    table, pool, _, _, q = batch
    home, s = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(home):
        attn = daa.BatchAttention(table, q.shape[1], pool)
        attn.plan()
    want, out, x = attn.run(q, stream=home), torch.zeros_like(q), torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=home):
        x.add_(1)
        attn.run(q, out=out, stream=s.cuda_stream if raw else s)
    s.synchronize()
    assert torch.equal(out, want)  # it ran, and not as part of the graph
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert not out.any() and x.tolist() == [1.0] * 4 and daa.device_error(reset=True) == 0
