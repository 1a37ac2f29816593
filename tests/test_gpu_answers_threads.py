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


@pytest.mark.parametrize("dtype,code", [(torch.float32, 2), (torch.bfloat16, 1), (torch.float16, 0)])
def test_draws_of_different_vocabularies(dtype, code):
    """Rows of other lengths take other amounts of shared memory: no call may take another's limit for its own."""
    sides = []
    for seed, V in enumerate((300, 24000, 120000, 9001)):
        x = (torch.randn(2, V, generator=torch.Generator().manual_seed(seed)) * 3).to(dtype).cuda()
        sides.append(dict(V=V, x=x, u=torch.tensor([0.3, 0.8]).cuda(), p=torch.full((2,), 0.9).cuda(), ids=torch.full((2,), -7, dtype=torch.int32).cuda(),
                          s=torch.cuda.Stream()))

    def call(d, stream):
        rv.sample(d["x"].data_ptr(), code, d["V"], 2, d["V"], None, None, d["p"].data_ptr(), None, d["u"].data_ptr(), d["ids"].data_ptr(), None, stream)

    torch.cuda.synchronize()
    for d in sides:
        call(d, None)
    torch.cuda.synchronize()
    want = [d["ids"].tolist() for d in sides]
    for d in sides:
        d["ids"].fill_(-7)
    torch.cuda.synchronize()
    raised = at_once([lambda i, d=d: call(d, d["s"].cuda_stream) for d in sides], 1500)
    assert not raised, raised[0]
    assert [d["ids"].tolist() for d in sides] == want


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
