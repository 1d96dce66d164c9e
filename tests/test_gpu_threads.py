"""Host threads that share torch's default stream: their calls are several launches each, which may alternate."""
import threading

import pytest
import torch

import lossless_draft_verification_online_amd as sdv
from cache_helpers import DEV, Batch
from test_gpu_sample import logits_of, place, uniforms

pytestmark = pytest.mark.gpu


def run_in_threads(calls, rounds=60):
    """Each call by its own thread, over and over; every result against the one that it gives alone."""
    want = [call() for call in calls]
    torch.cuda.synchronize()
    barrier = threading.Barrier(len(calls))
    got, failed = [[] for _ in calls], []

    def work(k):
        try:
            barrier.wait()
            for _ in range(rounds):
                got[k].append(calls[k]())
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for k, results in enumerate(got):
        for res in results:
            assert all(torch.equal(a, b) for a, b in zip(res, want[k]))


def test_sampling():
    calls = []
    for k in range(4):
        z, u = place(logits_of(6 + k, 40001, "bf16", k)), torch.tensor(uniforms(6 + k, k), device=DEV)
        p = torch.full((6 + k,), 900, dtype=torch.int32, device=DEV)

        def call(z=z, u=u, p=p):
            tok, prob, extra = sdv.sample(z, u, 0.9, top_p_milli=p, probs=True)
            return tok, prob, extra["kept_tokens"], extra["probs"]

        calls.append(call)
    run_in_threads(calls)


def test_attention_and_sampling():
    calls = []
    for k in range(3):
        b = Batch([k, 3], [3000 + 500 * k, 40], 2, 64, 16, "bf16", k, Hq=8)
        args = (b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV), *b.index_args())
        calls.append(lambda args=args: (sdv.attend(*args),))
    z, u = place(logits_of(5, 40001, "fp32", 9)), torch.tensor(uniforms(5, 9), device=DEV)
    calls.append(lambda: sdv.sample(z, u, 1.0)[:2])
    run_in_threads(calls)


def test_verification():
    calls = []
    for k in range(4):
        K, B, V = 3, 4 + k, 32000
        target, draft = place(logits_of(B * K + B, V, "bf16", 20 + k)), place(logits_of(B * K, V, "bf16", 30 + k))
        tok = torch.tensor([(7919 * (k + 1) * n) % V for n in range(B * K)], dtype=torch.int32, device=DEV)
        cu = torch.arange(0, B * K + 1, K, dtype=torch.int32, device=DEV)

        def call(target=target.contiguous(), draft=draft.contiguous(), tok=tok, cu=cu, k=k):
            return sdv.verify(target, draft, tok, cu, 1.0, k)[:2]

        calls.append(call)
    run_in_threads(calls)
