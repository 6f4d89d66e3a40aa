"""get_error from several host threads: a call waits for its own stream alone, and an error is
reported once."""
import threading
import time

import pytest
import torch

import lfm2_gated_short_gb300 as sc

pytestmark = pytest.mark.gpu


def test_an_idle_stream_is_not_held_up_by_a_busy_one():
    busy, idle = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (busy, idle):
        assert sc.get_error(stream=s) == 0
    sc.check_wait_limit(stream=busy)  # about 2 s, then DEV_TIMEOUT
    codes = []
    asker = threading.Thread(target=lambda: codes.append(sc.get_error(stream=busy)))
    asker.start()
    time.sleep(0.2)  # it is waiting for its stream now
    assert asker.is_alive()
    t = time.perf_counter()
    assert sc.get_error(stream=idle) == 0
    waited = time.perf_counter() - t
    still = asker.is_alive()
    asker.join()
    assert codes == [sc.DEV_TIMEOUT]
    assert still and waited < 0.5, waited
    assert sc.get_error() == 0


def test_more_threads_than_words_and_every_error_once():
    """100 threads ask 20 times each, on streams of their own, while one stream raises errors."""
    n, rounds = 100, 20
    pages = sc.page_cache(2, 2, 4)
    pool = torch.zeros((1, 4, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    bad = torch.tensor([9], dtype=torch.int32, device="cuda")
    length = torch.tensor([1], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    seen, failures = [[] for _ in range(n)], []

    def ask(j):
        try:
            s = torch.cuda.Stream()
            for _ in range(rounds):
                seen[j].append(sc.get_error(stream=s))
        except Exception as e:  # reported on the main thread
            failures.append(e)
    threads = [threading.Thread(target=ask, args=(j,)) for j in range(n)]
    for t in threads:
        t.start()
    sc.pages_resize(*pages, bad, length, pool, pool.clone())
    torch.cuda.synchronize()
    for t in threads:
        t.join()
    assert not failures
    codes = [c for s in seen for c in s] + [sc.get_error()]
    assert sorted(codes)[-2:] == [0, sc.DEV_BAD_SLOT], sorted(codes)[-5:]
