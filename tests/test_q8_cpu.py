"""The 8-bit KV cache's host side without a device: what the C entry points and
the Python class refuse before they touch a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from cross_model_shared_gb300 import QuantizedKVPool
from cross_model_shared_gb300 import _native as N
from cross_model_shared_gb300 import build as B
from cross_model_shared_gb300.q8 import _HostInts


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def config(**change):
    c = dict(num_pages=4, page_size=16, num_kv_heads=2, head_dim=64, max_batch=2, max_pages_per_seq=4, k_pages=0x1000,
             v_pages=0x2000, scales=0x3000, block_table=0x4000, seq_lens=0x5000, error_word=0x6000, initial_seq_lens=None)
    return N.shkv_q8_pool_config(**{**c, **change})


@pytest.mark.parametrize("change,status", [
    *[({f: 0}, "INVALID_ARG") for f in ("num_pages", "num_kv_heads", "max_batch", "max_pages_per_seq")],
    *[({f: None}, "INVALID_ARG") for f in ("k_pages", "v_pages", "scales", "block_table", "seq_lens", "error_word")],
    *[({f: 0x1008}, "INVALID_ARG") for f in ("k_pages", "v_pages", "scales")],
    ({"block_table": 0x4002}, "INVALID_ARG"),
    ({"page_size": 8}, "UNSUPPORTED"), ({"page_size": 64}, "UNSUPPORTED"), ({"head_dim": 32}, "UNSUPPORTED"),
    ({"head_dim": 256}, "UNSUPPORTED"), ({"max_batch": 1025}, "UNSUPPORTED"),
    ({"num_pages": 2 ** 31 // (2 * 16)}, "UNSUPPORTED"),                    # rows past 32 bits
    ({"max_pages_per_seq": 2 ** 27}, "UNSUPPORTED"),                         # lengths past 32 bits
])
def test_pools_that_cannot_be(lib, change, status):
    h = ctypes.c_void_p(7)
    assert lib.shkv_q8_pool_create(ctypes.byref(config(**change)), ctypes.byref(h)) == getattr(N, f"SHKV_ERR_{status}")
    assert not h.value


@pytest.mark.parametrize("lens", [[65, 0], [0, -1]])
def test_initial_lengths_outside_the_pool(lib, lens):
    a = np.array(lens, np.int32)
    h = ctypes.c_void_p()
    cfg = config(initial_seq_lens=a.ctypes.data)
    assert lib.shkv_q8_pool_create(ctypes.byref(cfg), ctypes.byref(h)) == N.SHKV_ERR_CAPACITY


def test_null_arguments(lib):
    bad = N.SHKV_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert lib.shkv_q8_pool_create(None, None) == bad
    assert lib.shkv_q8_pool_destroy(None) == bad
    assert lib.shkv_q8_pool_set_seq_lens(None, 1, None, None) == bad
    assert lib.shkv_q8_pool_get_seq_lens(None, 1, None) == bad
    assert lib.shkv_q8_check_errors(None, None, None) == bad
    assert lib.shkv_q8_append_kv(None, 1, None, None, None, 128, None, 128, None) == bad
    assert lib.shkv_q8_read_kv(None, 1, None, None, None, 128, None, 128, None) == bad
    assert lib.shkv_q8_workspace_size(None, ctypes.byref(n), ctypes.byref(n)) == bad
    assert lib.shkv_q8_decode_attention(None, 1, 1, 2, None, 1.0, None, None, None, 0, None) == bad
    assert lib.shkv_q8_chunk_attention(None, 1, None, 2, None, 128, 1.0, None, None, None, 0, None) == bad


def test_a_pool_on_the_cpu_is_refused(lib):
    with pytest.raises(ValueError):
        QuantizedKVPool(4, 16, 2, 64, 1, 4, device="cpu")


@pytest.mark.parametrize("x", [[3, 0, 5], (3, 0, 5), np.array([3, 0, 5]), np.array([3, 0, 5], np.int16)[::1],
                               np.array([3, 9, 0, 9, 5])[::2], torch.tensor([3, 0, 5]), range(3, 4)])
def test_host_integers(x):
    a = _HostInts(x, "x")
    want = list(x) if isinstance(x, range) else [3, 0, 5]
    assert a.n == len(want) and a.total == sum(want)
    assert list((ctypes.c_int32 * a.n).from_address(a.ptr)) == want


def test_no_integers():
    a = _HostInts([], "x")
    assert (a.n, a.total, a.ptr) == (0, 0, None)


@pytest.mark.parametrize("x", [[-1], [2 ** 31], [1.5], ["1"], [None], 3, np.array(3), np.zeros((2, 2), np.int32),
                               torch.zeros(2, 2, dtype=torch.int32), np.array([1.0]), [2 ** 70]])
def test_what_is_no_list_of_lengths(x):
    with pytest.raises(ValueError):
        _HostInts(x, "x")
