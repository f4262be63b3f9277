"""sparse_attn_paged_check_errors: the words of all kernels, and what a call costs."""
import ctypes
import statistics
import time

import pytest
import torch

import sparse_paged_attention_gb300 as spa
from workloads import latent_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def test_words_of_the_indexer_and_the_latent_kernels(dev):
    """Each kernel's flag is seen once, by the check after it, and none is left behind."""
    INDEX = spa.SPA_STATUS["SPA_ERR_INDEX"]
    inp = latent_inputs([20], 64, 16, 16, seed=65)
    rows, _ = inp.pool(False)
    pool = spa.LatentPool(rows.to(dev), inp.block_table.to(dev), 16)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=dev)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    far = i32(100000)
    keys = z(2, 8, 17, dt=torch.int32)
    calls = [
        lambda: spa.sparse_attn_latent_write(z(1, 64), z(1, 16), far, pool),
        lambda: spa.sparse_attn_latent_read(far, pool),
        lambda: spa.sparse_attn_latent_decode(z(1, 4, 64), z(1, 4, 16), pool, far, scale=1.0),
        lambda: spa.sparse_attn_latent_prefill(z(4, 2, 24), z(4, 2, 16), z(4, 8), z(4, 2, 16), i32(0, 5),
                                               i32(0, 4), scale=1.0),
        lambda: spa.sparse_attn_indexer_logits(z(1, 32, 128), z(1, 32, dt=torch.float32), keys, i32(7)[None],
                                               i32(63), ratio=4, num_cols=8),
    ]
    assert spa.sparse_attn_paged_check_errors() == 0
    for call in calls:
        call()
        assert spa.sparse_attn_paged_check_errors() == INDEX
        assert spa.sparse_attn_paged_check_errors() == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in calls:                               # all of them, on another stream, then one check of it
        with torch.cuda.stream(side):
            call()
    assert spa.sparse_attn_paged_check_errors(side) == INDEX
    assert spa.sparse_attn_paged_check_errors() == 0


def test_an_error_left_by_another_call_is_not_reported(dev):
    """A CUDA call of someone else that was refused (a copy of no such direction) is not the check's."""
    lib = spa.load_library()
    lib.cudaMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
    lib.cudaPeekAtLastError.argtypes, lib.cudaGetLastError.argtypes = [], []
    host = ctypes.c_int(0)
    refused = lib.cudaMemcpy(ctypes.addressof(host), ctypes.addressof(host), 4, 77)
    assert refused != 0 and lib.cudaPeekAtLastError() == refused
    try:
        assert spa.sparse_attn_paged_check_errors() == 0
        assert lib.cudaPeekAtLastError() == refused      # (nor is it taken away)
    finally:
        lib.cudaGetLastError()


def test_cost_does_not_grow_with_the_kernels(dev):
    """No more than a read and a clear of three words, as it was before the latent kernels (six small
    blocking copies; half more for the spread of such times, where a word each would take twice as long)."""
    lib = spa.load_library()
    lib.cudaMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    host = ctypes.c_int(0)

    def copies():
        for _ in range(3):
            assert lib.cudaMemcpy(ctypes.addressof(host), word.data_ptr(), 4, 2) == 0   # to the host
            assert lib.cudaMemcpy(word.data_ptr(), ctypes.addressof(host), 4, 1) == 0   # and back

    def us(f):
        times = []
        for _ in range(300):
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return statistics.median(times) * 1e6
    torch.cuda.synchronize()
    us(copies), us(spa.sparse_attn_paged_check_errors)
    six, check = (min(x) for x in zip(*[(us(copies), us(spa.sparse_attn_paged_check_errors))
                                        for _ in range(5)]))
    print(f"six copies {six:.1f} us, check_errors {check:.1f} us")
    assert check < 1.5 * six
