"""Calls from several host threads at once: what a call sets up for its kernel
(the shared memory that it may use) is not another call's."""
import threading

import pytest
import torch

import structured_sparse_quantized_b200 as ss

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def at_once(jobs, repeats):
    """Each job on a host thread and a stream of its own, `repeats` times, all
    at once; every result must be the job's own result alone."""
    wants = [job(None) for job in jobs]
    torch.cuda.synchronize()
    start, failures = threading.Barrier(len(jobs)), []

    def work(job, want):
        try:
            s = torch.cuda.Stream()
            start.wait()
            got = [job(s) for _ in range(repeats)]
            s.synchronize()
            for outs in got:
                for g, w in zip(outs, want):
                    assert torch.equal(g, w)
        except Exception as e:  # noqa: BLE001 (reported below, in the test's own thread)
            failures.append(repr(e))
    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[0]
    assert ss.ss_get_device_status() == ss.SS_OK


@pytest.mark.parametrize("pattern", ["6:8", "8:10"])
def test_norms_of_different_lengths(pattern):
    """Rows of lengths that one kernel serves, with different shared memory."""
    g = torch.Generator().manual_seed(1)
    jobs = []
    for K in (3080, 4096, 3600, 3200):
        X, w = torch.randn(1200, K, generator=g).to(BF).cuda(), torch.ones(K, device="cuda")
        jobs.append(lambda s, X=X, w=w: ss.norm_quant_lift_act(X, w, 1e-5, pattern, "int8", stream=s))
    at_once(jobs, 200)


def test_weights_of_different_lengths():
    g = torch.Generator().manual_seed(2)
    jobs = []
    for K in (12800, 32000, 16000, 24000):
        W = torch.randn(64, K, generator=g).cuda()
        jobs.append(lambda s, W=W: ss.compress_weight(W, "6:8", "int8", stream=s))
    at_once(jobs, 100)
