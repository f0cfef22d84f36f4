"""The 4-bit cache and the page pool on streams of the caller's: what a call reads,
and the memory it uses, belong to the stream that it names."""
import numpy as np
import pytest
import torch

import q4_support as ref

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


@pytest.fixture(autouse=True)
def no_device_error(daa):
    yield
    assert daa.device_error(reset=True) == 0


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _late_pool(daa, s):
    """A pool of 6 slots whose arrays are filled on stream s, behind other work; its state."""
    lens = [30, 16, 1, 0, 100, 0]
    st = {"seq_len": np.array(lens, np.int32), "held": np.array([-(-x // 16) for x in lens], np.int32),
          "block_table": np.full((6, 10), -1, np.int32)}
    free = list(range(39, -1, -1))
    for i, h in enumerate(st["held"]):
        st["block_table"][i, :h] = [free.pop() for _ in range(h)]
    st["free"] = free
    stack = np.full(40, -1, np.int32)
    stack[:len(free)] = free
    src = [_dev(x) for x in (st["seq_len"], st["held"], st["block_table"], stack, np.array([len(free), 0], np.int32))]
    dst = [torch.zeros_like(x) for x in src]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
        for d, x in zip(dst, src):
            d.copy_(x)
    return daa.PagePool.from_tensors(*dst), st


def _same_host(pool, st):
    assert np.array_equal(pool.h_len, st["seq_len"]) and np.array_equal(pool.h_held, st["held"])
    assert pool.h_free == len(st["free"])


@pytest.mark.parametrize("raw", [False, True])
def test_lengths_are_read_on_the_stream_of_the_call(daa, raw):
    s = torch.cuda.Stream()
    name = s.cuda_stream if raw else s
    pool, st = _late_pool(daa, s)
    slots, new = [4, 0, 3], [1, 40, 17]
    t = pool.step(slots, new, stream=name)
    want = ref.step_table(st, slots, new, True)
    torch.cuda.synchronize()
    for n, w in want.items():
        assert np.array_equal(getattr(t, n).cpu().numpy(), w), n
    _same_host(pool, st)
    pool, st = _late_pool(daa, s)
    pool.set_lengths([0, 4], [17, 100], stream=name)
    st["seq_len"][[0, 4]] = [17, 100]
    torch.cuda.synchronize()
    assert np.array_equal(pool.seq_len.cpu().numpy(), st["seq_len"])
    _same_host(pool, st)
    pool, st = _late_pool(daa, s)
    pool.release([0, 4], stream=name)
    torch.cuda.synchronize()
    assert pool.counters.tolist() == [pool.h_free, 0] and pool.h_free == len(st["free"]) + 9


def _chunk(daa, hq=32, hkv=8, d=128, cached=3001, new=700):
    """A chunk whose workspace is large (its pages in bf16): more than 10 MB, so a block of its own."""
    rng = np.random.default_rng(1)
    t, n = ref.make_table(rng, [cached, 20], [new, 1])
    pool = np.concatenate([rng.integers(0, 256, (n, hkv, 2, 8 * d), dtype=np.uint8),
                           rng.integers(40, 64, (n, hkv, 2, d), dtype=np.uint8)], -1)
    table = daa.PageTable.from_host(*(t[x] for x in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len")), DEV)
    q = torch.from_numpy(rng.standard_normal((new + 1, hq, d))).bfloat16().to(DEV)
    return table, _dev(pool), q


def test_workspace_outlives_its_object(daa):
    """An object dropped while its run is under way: its workspace is nobody else's until the run has ended."""
    table, pages, q = _chunk(daa)
    want = daa.BatchAttentionQ4(table, q.shape[1], pages).run(q)
    out, s = torch.empty_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        attn = daa.BatchAttentionQ4(table, q.shape[1], pages)
        n, at = attn.workspace.numel(), attn.workspace.data_ptr()
        assert n > 10 << 20
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        attn.run(q, out=out, stream=stream)
        pending = not s.query()
        del attn
        other = torch.empty(n, dtype=torch.uint8, device=DEV)  # never written
        # not this memory, or on a stream that waits for the run
        safe = other.data_ptr() != at or not torch.cuda.current_stream().query()
        s.synchronize()
        assert pending and safe
        assert torch.equal(out, want)
        del other
        torch.cuda.synchronize()


def test_workspace_waits_for_what_its_memory_was(daa):
    """A workspace in memory that the constructor's stream still writes for a tensor freed before."""
    table, pages, q = _chunk(daa)
    attn = daa.BatchAttentionQ4(table, q.shape[1], pages)
    want = attn.run(q)
    n, head = attn.workspace.numel(), attn.workspace[:256].clone()  # of the plan
    del attn
    s = torch.cuda.Stream()
    before = torch.empty(n, dtype=torch.uint8, device=DEV)
    at = before.data_ptr()
    before.fill_(7)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    before.fill_(7)
    del before
    attn = daa.BatchAttentionQ4(table, q.shape[1], pages)
    assert attn.workspace.data_ptr() == at and not torch.cuda.current_stream().query()
    attn.plan(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(attn.workspace[:256], head)
    out = attn.run(q, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("raw", [False, True])
def test_pool_outlives_its_object(daa, raw):
    """A pool dropped while a call on it is under way on another stream: its arrays are nobody else's until that has ended."""
    s = torch.cuda.Stream()
    i32 = dict(dtype=torch.int32, device=DEV)
    pool = daa.PagePool(1000, 50, 70_000)
    n, at = pool.block_table.numel(), pool.block_table.data_ptr()
    a = (torch.tensor([3], **i32), torch.tensor([20], **i32), *(torch.empty(2, **i32) for _ in range(3)), torch.empty(1, **i32))
    for busy in (0, BUSY):  # a first kernel call may wait for the device
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(busy)
        pool.build(*a, stream=s.cuda_stream if raw else s)
    pending = not s.query()
    del pool
    other = torch.empty(n, **i32)  # never written
    # not this memory, or on a stream that waits for the call
    safe = other.data_ptr() != at or not torch.cuda.current_stream().query()
    s.synchronize()
    assert pending and safe
    assert a[2].tolist() == [0, 20] and a[3].tolist() == [0, 2] and a[4].tolist() == [0, 1]


def test_steps_of_two_pools_in_two_threads(daa):
    """Steps of different sizes prepared at the same time: neither changes what the other is launched with."""
    import threading
    failed, go = [], threading.Barrier(2)

    def work(batch):
        try:
            s = torch.cuda.Stream()
            pool = daa.PagePool(2 * batch, batch, 4)
            i32 = dict(dtype=torch.int32, device=DEV)
            a = (torch.arange(batch, **i32), torch.ones(batch, **i32), torch.empty(batch + 1, **i32),
                 torch.empty(batch + 1, **i32), torch.empty(batch, **i32), torch.empty(batch, **i32))
            torch.cuda.synchronize()
            go.wait()
            for _ in range(3000):
                pool.build(*a, stream=s)
            s.synchronize()
            assert a[3][-1] == batch
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(b,)) for b in (2500, 8000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
