"""The page bookkeeping calls' host-side checks (CPU only: no call here
reaches the GPU) and hand cases of their oracle."""
import numpy as np
import pytest
import torch

import oracle

A = 1 << 12  # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verify_mla_gb300 import build as B
    B.build()
    from speculative_decoding_verify_mla_gb300 import load_library
    return load_library()


def test_workspace_query(lib):
    f = lib.sv_kv_pages_workspace_bytes
    assert f(0, 0, 0) >= 256 and f(-1, 2, 2) == 256
    assert f(1000, 8, 4) >= f(1000, 8, 0) >= f(100, 8, 0) > 0
    assert f(2**31 - 1, 16, 16) > 2**33  # sizes past 32 bits


def test_copy_checks(lib):
    f = lib.kv_pages_copy
    ok = [A, 8, A, 8, 1, 65536, A, A, 4, None, None]

    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[int(k[1:])] = v
        return f(*args)
    assert call(_8=0) == 0 and call(_4=0) == 0 and call(_5=0) == 0        # nothing to do
    assert call(_8=-1) == 2 and call(_1=-1) == 2 and call(_3=-1) == 2 and call(_4=-1) == 2
    assert call(_5=65535) == 5 and call(_5=(1 << 30) + 16) == 5           # page bytes
    for i in (0, 2, 6, 7):
        assert call(**{f"_{i}": None}) == 1
    assert call(_0=A + 8) == 3 and call(_2=A + 4) == 3 and call(_6=A + 2) == 3 and call(_7=A + 1) == 3


def _resize_args():
    return [A, 64, 64, A, A, 4, 8, A, A, A, A, A, 1 << 20, None, None]


def test_resize_checks(lib):
    f = lib.kv_pages_resize

    def call(**kw):
        args = _resize_args()
        for k, v in kw.items():
            args[int(k[1:])] = v
        return f(*args)
    assert call(_1=0) == 2 and call(_5=-1) == 2 and call(_6=-1) == 2
    assert call(_2=32) == 5
    assert call(_5=1 << 20, _6=1 << 12) == 2 and call(_5=1, _6=1 << 26) == 2  # 2^31 entries, 2^31 positions
    for i in (0, 3, 4, 7, 8, 9, 10):
        assert call(**{f"_{i}": None}) == 1
        assert call(**{f"_{i}": A + 2}) == 3
    assert call(_11=None) == 4 and call(_12=64) == 4 and call(_11=A + 16) == 3
    assert call(_6=0, _4=None) == 1  # no entries, but lengths


def test_most_requests(lib):
    assert lib.kv_pages_resize(*[A, 64, 64, A, A, (1 << 30) + 1, 1, A, A, A, A, A, 1 << 40, None, None]) == 2
    fork = [A, 64, 64, 2, 1024, A, A, A, 4, 8, A, A, (1 << 30) + 1, A, A, A, A, 1 << 40, None, None]
    assert lib.kv_pages_fork(*fork) == 2
    fork[8:10], fork[12] = [(1 << 30) + 1, 1], 2
    assert lib.kv_pages_fork(*fork) == 2


def test_fork_and_compact_checks(lib):
    ok = [A, 64, 64, 2, 1024, A, A, A, 4, 8, A, A, 2, A, A, A, A, 1 << 20, None, None]

    def fork(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[int(k[1:])] = v
        return lib.kv_pages_fork(*args)
    assert fork(_1=0) == 2 and fork(_8=-1) == 2 and fork(_12=-1) == 2 and fork(_3=0) == 2 and fork(_4=0) == 2
    assert fork(_8=0) == 2 and fork(_9=0) == 2  # forks among no requests
    assert fork(_2=16) == 5 and fork(_4=1000) == 5 and fork(_4=(1 << 24) + 16) == 2
    for i in (0, 5, 6, 7, 10, 11, 13, 14, 15):
        assert fork(**{f"_{i}": None}) == 1
    assert fork(_0=A + 8) == 3 and fork(_10=A + 2) == 3
    assert fork(_16=None) == 4 and fork(_17=8) == 4 and fork(_16=A + 64) == 3
    ok2 = [A, 64, 64, 2, 1024, A, A, A, 4, 8, A, A, A, A, A, 1 << 20, None, None]

    def compact(**kw):
        args = list(ok2)
        for k, v in kw.items():
            args[int(k[1:])] = v
        return lib.kv_pages_compact(*args)
    assert compact(_1=0) == 2 and compact(_3=0) == 2 and compact(_9=-1) == 2
    assert compact(_2=65) == 5 and compact(_4=24) == 5
    for i in (0, 5, 6, 7, 10, 11, 12, 13):
        assert compact(**{f"_{i}": None}) == 1
    assert compact(_14=None) == 4 and compact(_15=0) == 4


def test_binding_refuses_before_the_library(lib):
    import speculative_decoding_verify_mla_gb300 as sv
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros((4, 64, 512), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.kv_pages_copy(pool, pool, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        sv.kv_pages_resize(i, torch.zeros((4, 2), dtype=torch.int32), i, i)


def test_oracle_resize_by_hand():
    refs = np.array([1, 0, 2, 1, 0, 0], np.int32)
    table = np.array([[2, 0, -7], [2, 3, -7], [-7, -7, -7]], np.int32)
    lens = np.array([100, 128, 0], np.int32)
    # 0 drops its second page, 1 grows past its two full pages, 2 is admitted with one
    r, t, n, st = oracle.ref_pages_resize(refs, table, lens, np.array([64, 129, 10], np.int32))
    assert st == 0 and r.tolist() == [1, 1, 2, 1, 0, 0] and n.tolist() == [64, 129, 10]
    assert t.tolist() == [[2, -1, -7], [2, 3, 0], [1, -7, -7]]
    # a partly filled page that two requests hold cannot be grown into
    r, t, n, st = oracle.ref_pages_resize(refs, table, np.array([60, 128, 0], np.int32), np.array([61, -1, 0], np.int32))
    assert st == 0x10 and n.tolist() == [60, 128, 0]
    # too few pages: the first request that does not fit and those after it that need some keep their lengths
    r, t, n, st = oracle.ref_pages_resize(np.array([1, 1, 1], np.int32), np.array([[0, -1], [1, 2]], np.int32),
                                          np.array([64, 128], np.int32), np.array([128, 64], np.int32))
    assert st == 0 and t.tolist() == [[0, 2], [1, -1]]
    r, t, n, st = oracle.ref_pages_resize(np.array([1, 1, 1], np.int32), np.array([[0, -1], [1, 2]], np.int32),
                                          np.array([64, 128], np.int32), np.array([128, -1], np.int32))
    assert st == 0x20 and n.tolist() == [64, 128] and r.tolist() == [1, 1, 1]


def test_oracle_fork_and_compact_by_hand():
    pool = np.arange(6 * 64 * 16, dtype=np.uint8).reshape(1, 6, 64, 16)
    refs = np.array([0, 1, 0, 1, 0, 0], np.int32)
    table = np.array([[3, 1], [-1, -1], [-1, -1]], np.int32)
    p2, r, t, n, st = oracle.ref_pages_fork(pool, refs, table, np.array([66, 0, 0], np.int32), [0, 0], [2, 1])
    assert st == 0 and r.tolist() == [1, 1, 1, 3, 0, 0] and n.tolist() == [66, 66, 66]
    assert t.tolist() == [[3, 1], [3, 2], [3, 0]]
    assert np.array_equal(p2[0, 0, :2], pool[0, 1, :2]) and np.array_equal(p2[0, 0, 2:], pool[0, 0, 2:])
    p3, r, t, m, live, st = oracle.ref_pages_compact(pool, refs, table, np.array([66, 0, 0], np.int32))
    assert live == 2 and st == 0 and m.tolist() == [-1, 1, -1, 0, -1, -1] and t[0].tolist() == [0, 1]
    assert np.array_equal(p3[0, 0], pool[0, 3]) and np.array_equal(p3[0, 3], pool[0, 3]) and r.tolist() == [1, 1, 0, 0, 0, 0]
