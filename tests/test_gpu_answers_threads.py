"""Calls of several host threads at once, each with its own stream and memory."""
import threading

import pytest
import torch

import token_level_early_gb300 as rv
from test_gpu_kv8_copy import bits, random_cache

pytestmark = pytest.mark.gpu


def at_once(jobs, rounds):
    """Every job's call `rounds` times in a thread of its own; what they raised."""
    start, raised = threading.Barrier(len(jobs)), []

    def work(job):
        start.wait()
        try:
            for i in range(rounds):
                job(i)
        except Exception as e:
            raised.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def test_copies_of_different_numbers_of_pairs():
    sides = []
    for n in (1, 7, 40, 300):
        c = random_cache(n, n + 1, 1, 64, 100, 16)
        f, t, m = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0] * n, list(range(1, n + 1)), [100] * n))
        sides.append(dict(n=n, c=c, f=f, t=t, m=m, s=torch.cuda.Stream()))
    torch.cuda.synchronize()
    raised = at_once([lambda i, d=d: rv.kv8_copy(d["c"].c, d["c"].c, d["n"], d["f"].data_ptr(), d["t"].data_ptr(), d["m"].data_ptr(), d["c"].err.data_ptr(),
                                                 d["s"].cuda_stream) for d in sides], 1500)
    assert not raised, raised[0]
    for d in sides:
        assert int(d["c"].err) == 0
        for x in d["c"].tail:
            y = bits(x)
            assert (y[1:] == y[:1]).all()
        for x in d["c"].codes:
            y = bits(x)[:, :, :100]
            assert (y[1:] == y[:1]).all()
