"""Limits that the history layer's header, binding and definition share (CPU)."""
import os
import re

import numpy as np

from dlrm_sparse_embedding_amd import emb as E
from oracle import history_oracle as H

HEADER = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "emb.h")).read()


def test_the_entry_that_hides():
    value = float(re.search(r"#define EMB_HIDDEN_BIAS \((-[\d.]+)f\)", HEADER).group(1))
    assert value == E.EMB_HIDDEN_BIAS == H.HIDDEN
    # masks in use are below it, and weights made from scores above it are right to half a step of bf16
    assert max(-1e4, -65504.0, -1e9) <= value and 6 * 2.0 ** -24 * -value <= 2.0 ** -8


def test_the_definition_hides_from_it_down():
    q, k, v = (np.ones((2, 1, 4)) for _ in range(3))
    for entry, seen in ((E.EMB_HIDDEN_BIAS, False), (np.nextafter(E.EMB_HIDDEN_BIAS, 0.0), True), (-1e4, False)):
        out, lse, _ = H.attention(q, k, v, [0, 2], 1.0, True, np.array([[entry], [entry]]), (2, 2, 0))
        assert (out == (1 if seen else 0)).all() and np.isfinite(lse).all() == seen
