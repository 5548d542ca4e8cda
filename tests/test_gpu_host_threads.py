"""Two host threads that call on one stream at once: every result is the one the
same call gives alone, bit for bit."""
import threading

import pytest
import torch

from dense_fp32_gemm_f32_amd import binding

pytestmark = pytest.mark.gpu


def _calls(seed):
    """Calls that pass partial sums through the stream's workspace: adapters of
    few rows, sliced gradients of both kinds, and adapters of many rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    few, many = 24 + seed, 130 + seed
    args = {}
    for m in (few, many):
        index = torch.randint(-1, 3, (m,), generator=g, device="cuda").to(torch.int32)
        offsets, order, _ = binding.group_rows(index, 3)
        args[m] = (rand(m, 1024), rand(256, 1024), rand(3, 8, 1024), rand(3, 256, 8), offsets,
                   order)
    rows = 1500
    spans = torch.tensor([0, 700, rows], dtype=torch.int32, device="cuda")
    a, b, thin = rand(rows, 100), rand(rows, 140), rand(rows, 12)
    return [lambda: binding.gemm_adapters(*args[few], trans=True)[0],
            lambda: binding.gemm_grouped_wgrad(a, b, spans),
            lambda: binding.gemm_grouped_wgrad(thin, b, spans),
            lambda: binding.gemm_adapters(*args[many], trans=True)[0]]


@pytest.mark.parametrize("side", [False, True])
def test_two_threads_on_one_stream(gpu_lib, side):
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    calls = [_calls(seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        alone = [[call() for call in per] for per in calls]
    torch.cuda.synchronize()
    results, errors = [[], []], []
    start = threading.Barrier(2, timeout=60)

    def work(t):
        try:
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(20):
                    results[t].append([call() for call in calls[t]])
        except BaseException as e:   # reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for t in range(2):
        assert len(results[t]) == 20
        for got in results[t]:
            for x, y in zip(got, alone[t]):
                assert torch.equal(x, y)
