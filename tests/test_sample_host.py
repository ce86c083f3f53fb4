"""sample_tokens: host-side checks (CPU only: no call here reaches the GPU) and
hand cases of its oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle

A = 1 << 12
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verify_mla_gb300 import build as B
    B.build()
    from speculative_decoding_verify_mla_gb300 import load_library
    return load_library()


def test_checks(lib):
    ok = [A, 0, 4, 1000, 1000, A, None, 1.0, None, 0, None, 1.0, None, 0.0, A, None, None, None]

    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[int(k[1:])] = v
        return lib.sample_tokens(*args)
    assert call(_2=0) == 0
    assert call(_2=-1) == 2 and call(_3=0) == 2 and call(_4=999) == 2 and call(_2=1 << 30) == 2
    assert call(_1=2) == 5 and call(_3=(1 << 22) + 1, _4=1 << 23) == 5
    assert call(_7=math.nan) == 2 and call(_7=math.inf) == 2 and call(_11=math.nan) == 2 and call(_13=math.nan) == 2
    for i in (0, 5, 14):
        assert call(**{f"_{i}": None}) == 1
        assert call(**{f"_{i}": A + 2}) == 3
    assert call(_1=1, _0=A + 1) == 3
    for i in (6, 8, 10, 12, 15):
        assert call(**{f"_{i}": A + 2}) == 3


def test_binding_refuses_before_the_library(lib):
    import speculative_decoding_verify_mla_gb300 as sv
    x, u = torch.zeros((2, 8)), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        sv.sample_tokens(x, u)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        sv.sample_tokens(x.half(), u)
    with pytest.raises(ValueError):
        sv.sample_tokens(x[0], u)


def test_oracle_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.25, 0.05]))
    f = oracle.ref_sample_row
    assert [f(x, u)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.94, 0.96, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3, 4, 4]
    tok, p = f(x, 0.99, top_k=2)[:2]
    assert tok == 3 and np.allclose(p, [0, 0.4 / 0.65, 0, 0.25 / 0.65, 0])
    tok, p = f(x, 0.0, top_p=0.7)[:2]          # 0.4 + 0.25 < 0.7 <= + 0.2
    assert tok == 1 and np.count_nonzero(p) == 3
    assert np.count_nonzero(f(x, 0.0, min_p=0.45)[1]) == 3   # 0.4, 0.25, 0.2 of a largest of 0.4
    assert np.count_nonzero(f(x, 0.0, top_k=3, top_p=0.45)[1]) == 1  # 0.4 of 0.85 is the share of the largest
    assert f(x, 0.9, temperature=0.0)[0] == 1 and f(x, 0.9, top_p=0.0)[0] == 1
    tied = np.array([1.0, 2.0, 2.0, 0.0])
    assert f(tied, 0.6, top_k=1)[0] == 2 and f(tied, 0.4, top_k=1)[0] == 1  # ties at the border stay
    assert f(np.full(4, -np.inf), 0.5)[0] == -1 and f(np.array([np.nan, 1.0]), 0.5)[0] == 1
    # low temperatures sharpen: 0.4^2 of the sum of squares
    assert np.isclose(f(x, 0.5, temperature=0.5)[1][1], 0.16 / (0.01 + 0.16 + 0.04 + 0.0625 + 0.0025))
