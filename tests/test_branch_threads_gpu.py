"""Beam selection and the paged cache's upkeep called by several host threads with different sizes: what a
launch needs of its kernel does not depend on what another thread's last call needed."""
import threading

import pytest
import torch

from oracle import branch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def index(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def in_threads(works, turns):
    """Each work's calls in a thread and on a stream of its own; returns what was raised."""
    errors, gate = [], threading.Barrier(len(works))
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()

    def body(work, stream):
        try:
            with torch.cuda.stream(stream):
                gate.wait(60)
                for _ in range(turns):
                    work()
        except Exception as e:  # handed to the test
            errors.append(e)
    threads = [threading.Thread(target=body, args=x) for x in zip(works, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("sizes", [(2000, 16384), (1300, 1500), (1229, 12288, 6000)])
def test_tables_of_different_heights_forked_by_threads(cuda_lib, sizes):
    """Turns are even, so that a table whose rows are exchanged in pairs ends as it began."""
    caches, works = [], []
    for B in sizes:
        o = branch.Cache([[2 * b, -1 if b % 3 else 2 * b + 1] for b in range(B)],
                         [1 if e % 2 == 0 or e // 2 % 3 == 0 else 0 for e in range(2 * B)], 8)
        table, refs = index(o.table), index(o.refs)
        parents = [b ^ 1 if b ^ 1 < B else b for b in range(B)]
        par = index(parents)
        caches.append((o, table, refs, parents, par))
        works.append(lambda t=table, p=par, r=refs: cuda_lib.paged_fork(t, p, r))
    assert in_threads(works, 400) == []
    assert cuda_lib.sync_status() == 0
    for o, table, refs, parents, par in caches:
        assert table.tolist() == o.table and refs.tolist() == o.refs
        cuda_lib.paged_fork(table, par, refs)
        o.fork(parents)
        assert cuda_lib.sync_status() == 0
        assert table.tolist() == o.table and refs.tolist() == o.refs


@pytest.mark.parametrize("sizes", [(2500, 3000, 2100, 2700), (5000, 16384, 5600, 4800)])
def test_batches_of_different_heights_reserved_by_threads(cuda_lib, sizes):
    """A page for each sequence the first time, nothing from then on."""
    caches, works = [], []
    for B in sizes:
        o = branch.Cache([[-1, -1] for _ in range(B)], [0] * (8 * B + 5), 8)
        table, refs = index(o.table), index(o.refs)
        lens = [1 + b % 11 for b in range(B)]
        kv = index(lens)
        caches.append((o, table, refs, lens))
        works.append(lambda t=table, n=kv, r=refs: cuda_lib.paged_reserve(t, n, r, 8))
    assert in_threads(works, 2000) == []
    assert cuda_lib.sync_status() == 0
    for o, table, refs, lens in caches:
        o.reserve(lens, list(range(len(lens) + 1)))
        assert table.tolist() == o.table and refs.tolist() == o.refs


def test_requests_of_different_widths_selected_by_threads(cuda_lib):
    """Up to 128 pieces in one launch: the lists that its blocks keep are of different sizes."""
    calls, works = [], []
    for W, V in ((128, 4096), (118, 4000), (113, 2048), (128, 300)):
        x = torch.randn(1, W, V, generator=torch.Generator(device=DEV).manual_seed(W + V), device=DEV)
        s = -torch.rand(1, W, generator=torch.Generator(device=DEV).manual_seed(W), device=DEV)
        assert cuda_lib.beam_select_workspace_bytes(1, W, V, 128) == 0
        want = [t.clone() for t in cuda_lib.beam_select(x, s, k=128)]
        last = [None]

        def work(x=x, s=s, last=last):
            last[0] = cuda_lib.beam_select(x, s, k=128)
        calls.append((want, last))
        works.append(work)
    assert in_threads(works, 300) == []
    assert cuda_lib.sync_status() == 0
    for want, last in calls:
        assert all(torch.equal(a, b) for a, b in zip(last[0], want))
