"""Ragged steps on the GPU: the attention of new tokens over the paged cache,
causal and windowed, against its definition in 64 bits; the request tables
against a plain count; slots, and the whole step of a ragged layer."""

import math

import pytest
import torch

from mla_latent_kv_39_b200 import Cache, Config, MLAError, abi, check_device_error, mla_get_device_error

from ragged_cases import TINY, V3, Ragged

pytestmark = pytest.mark.gpu

# (cached, new, padding): single rows, page and tile borders, ragged chunks with
# sequences that bring nothing, tokens cut over many workers, more tokens than workers
BATCHES = [
    ([0], [1], 0),
    ([1], [1], 3),
    ([62], [3], 0),
    ([255], [2], 1),
    ([256, 0, 64], [1, 5, 0], 2),
    ([0, 700, 63, 64, 1], [70, 1, 0, 33, 2], 5),
    ([9000], [1], 0),
    ([3000, 20], [2, 1], 0),
    ([200] * 40, [0, 1, 2, 3] * 10, 7),
]


@pytest.mark.parametrize("cached,new,pad", BATCHES)
def test_chunk_attention(cached, new, pad):
    r = Ragged(Config(**V3), cached, new, pad)
    r.run()
    check_device_error()
    r.check()


WINDOWS = [(1, 0), (1, 200), (17, 5), (62, 64), (63, 1), (64, 0), (65, 70), (300, 4), (256, 128), (10 ** 9, 3),
           (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_attention(window, sinks):
    r = Ragged(Config(**V3), [0, 700, 63, 64, 1500], [70, 1, 0, 33, 3], 5)
    r.run(window, sinks)
    check_device_error()
    r.check(window, sinks)
