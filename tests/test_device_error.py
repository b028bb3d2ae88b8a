"""Reading the device error word: what several kernel files have recorded is reported once, the first of them, and all
of it is cleared; and the call costs about what reading one word does, however many files there are."""
import time

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _bad_write(stream=None):
    """A cache row outside the cache: skipped and recorded."""
    k = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((1, 1, 64, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([64], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    api.dsa_kv_write(k, k, slots, cache, torch.zeros_like(cache), stream=stream)
    return cache


def _bad_pages(stream=None):
    """A request that asks for a page of an empty stack: refused and recorded."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = [i32(1), i32(0), i32(-1).view(1, 1), i32(0), i32(0), i32(0, 0), i32(0)]
    torch.cuda.synchronize()
    api.dsa_pages_update(*args, stream=stream)
    return args


def test_errors_of_several_files_are_read_once():
    assert api.dsa_get_device_error() == 0
    for calls in ((_bad_write,), (_bad_pages,), (_bad_write, _bad_pages), (_bad_pages, _bad_write, _bad_write)):
        keep = [call() for call in calls]
        assert api.dsa_get_device_error() == 5, calls
        assert api.dsa_get_device_error() == 0, calls
        del keep


def test_errors_of_another_stream():
    stream = torch.cuda.Stream()
    keep = _bad_write(stream=stream)
    assert api.dsa_get_device_error(stream) == 5
    assert api.dsa_get_device_error(stream) == 0 and api.dsa_get_device_error() == 0
    del keep


def _us(call, n=200):
    times = []
    for _ in range(9):
        t = time.perf_counter()
        for _ in range(n):
            call()
        times.append((time.perf_counter() - t) / n * 1e6)
    return sorted(times)[4]


def test_the_cost_of_reading_them():
    """Less than five reads of a word: it is a launch, a read, and the host's part.  (A read a file would be eleven.)"""
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    word.item(), api.dsa_get_device_error()
    assert _us(api.dsa_get_device_error) < 5 * _us(word.item)
