"""Serving operators without a GPU: refusals and oracle pins of states that an
ordinary batch does not have (each refusal returns before any CUDA work)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import serving as S
from query_adaptive_chunk_b200 import build as B


@pytest.fixture(scope="module")
def csa():
    if not os.path.exists(B.LIB) or any(os.path.getmtime(s) > os.path.getmtime(B.LIB)
                                        for s in B.sources()):
        B.build()
    from query_adaptive_chunk_b200 import csa as mod
    return mod


INVALID, UNSUPPORTED = 1, 2


def test_compress_of_a_paused_sequence_by_hand():
    """Position 9 is the last one, so 8 and 9 are local; 3 is the heaviest other."""
    w = np.array([[[0.0, 5.0, 1.0, 0.0, 2.0]]])
    pos = np.array([[[8, 3, 4, 9, 5]]])
    assert S.cache_compress(w, [5], 3, 0, 2, pos, [-1]) == [[[0, 1, 3]]]
    assert S.cache_compress(w, [5], 3, 0, 2, pos, [10]) == [[[0, 1, 3]]]
    assert S.cache_compress(w, [5], 3, 0, 2, None, [-1]) == [[[1, 3, 4]]]
