"""The calls over a cache in 8 bits and the pages' call from several host threads, on streams other than the current one's default, and
with a workspace of the caller's."""
import threading

import numpy as np
import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache8_helpers import DEV, Batch8, host
from test_gpu_kv_cache import freq
from test_gpu_pages import Pages

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream():
    """Each thread's calls are several launches that hand each other results: the threads' launches may alternate."""
    batches = [Batch8([4, 0, 2], [3000 + 100 * k, 50, 30], 2, 128, 16, 16, "bf16", k, Hq=8) for k in range(4)]
    want = [b.attend() for b in batches]
    tables = [Pages([3, 2, 9] * 40, [40, 100, 77] * 40, 16, k, spare=400) for k in range(4)]
    for p in tables:
        p.start = [x.clone() for x in p.args()]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        b, p = batches[k], tables[k]
        for step in range(30):
            got = b.attend()
            a = [x.clone() for x in p.start]
            placed, slots = sdv.kv_pages(a[0], a[1], a[2], p.n_d, a[3], a[4], 16)
            if step == 0:
                first = (placed.clone(), slots.clone(), a[0].clone())
            if not torch.equal(got, want[k]) or not all(torch.equal(x, y) for x, y in zip(first, (placed, slots, a[0]))):
                bad.append((k, step))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_another_stream():
    """Work goes on the current stream: what it waits for there is waited for."""
    b = Batch8([4, 0, 20], [300, 50, 7], 2, 128, 16, 16, "bf16", 18, Hq=4)
    caches = b.caches()
    table, length, cu = b.index_args()
    b.append(caches, freq(128).to(DEV))
    want = sdv.attend(b.q.to(DEV), caches[0], caches[1], table, length, cu, key_scales=caches[2], value_scales=caches[3])
    k, v, q, f = b.k.to(DEV), b.v.to(DEV), b.q.to(DEV), freq(128).to(DEV)
    again = b.caches()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the caches come late
        late = [torch.zeros_like(x.view(torch.uint8)).view(x.dtype) for x in again]
        for x, y in zip(late, again):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        sdv.kv_append(k, v, late[0], late[1], table, length, cu, key_scales=late[2], value_scales=late[3], inv_freq=f)
        out = sdv.attend(q, late[0], late[1], table, length, cu, key_scales=late[2], value_scales=late[3])
    side.synchronize()
    assert torch.equal(out, want)
    for x, y in zip(late, caches):
        assert np.array_equal(host(x), host(y))


def test_a_workspace_of_the_callers():
    b = Batch8([4, 0, 2], [3000, 50, 30], 2, 128, 16, 16, "bf16", 3, Hq=8)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(b.attend(workspace=ws), b.attend())
    p = Pages([3, 2, 9], [40, 100, 77], 16, 6, spare=20)
    a, c = p.args(), p.args()
    got = sdv.kv_pages(a[0], a[1], a[2], p.n_d, a[3], a[4], 16, workspace=ws)
    want = sdv.kv_pages(c[0], c[1], c[2], p.n_d, c[3], c[4], 16)
    assert all(torch.equal(x, y) for x, y in zip((*a, *got), (*c, *want)))


def test_results_in_given_tensors():
    b = Batch8([2, 5], [30, 7], 2, 64, 16, 8, "fp32", 4, Hq=4)
    out = torch.empty_like(b.q, device=DEV)
    assert b.attend(out=out) is out and torch.equal(out, b.attend())
    p = Pages([3, 2], [30, 7], 4, 16, spare=20)
    a = p.args()
    placed, slots = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(7, dtype=torch.int64, device=DEV)
    got = sdv.kv_pages(a[0], a[1], a[2], p.n_d, a[3], a[4], 4, placed=placed, slots=slots)
    assert got[0].data_ptr() == placed.data_ptr() and got[1].data_ptr() == slots.data_ptr() and placed.tolist() == [1, 1]
