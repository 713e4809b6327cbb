"""The range of the attention over INT4 rows: its scores are held times 2^-40, so a
scale whose factor 2^40 log2(e) scale is not finite is refused; over bf16 rows it is not."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def dsa():
    import dsa_indexer_indexshare_gb300 as m
    return m


def _call(dsa, name, scale, dt=2):
    """Status of a call whose workspace is too small: the arguments are checked before it."""
    b = ctypes.byref(dsa._Batch(1, 4, 4, 256, FAKE, FAKE, FAKE))
    if name == "rows":
        return dsa.lib.dsa_sparse_mla_attn_rows(FAKE, FAKE, FAKE, 100, dt, FAKE, 64, 16, scale, b, FAKE, None,
                                                FAKE, 128, None)
    f = {2: dsa.lib.dsa_sparse_mla_attn_int4kv, 0: dsa.lib.dsa_sparse_mla_attn}[dt]
    return f(FAKE, FAKE, FAKE, 100, FAKE, 64, 16, scale, b, FAKE, None, FAKE, 128, None)


@pytest.mark.parametrize("name", ["attn", "rows"])
def test_scales_that_overflow_are_refused(dsa, name):
    under = 2.0 ** 87 * (1 - 2.0 ** -24)  # the largest fp32 below 2^87
    for s in (2.0 ** 87, -2.0 ** 87, 1e38, float("inf"), -float("inf")):
        assert _call(dsa, name, s) == dsa.DSA_ERR_UNSUPPORTED, s
        assert b"2^87" in dsa.lib.dsa_last_error_string()
        assert _call(dsa, name, s, dt=0) == dsa.DSA_ERR_WORKSPACE  # (bf16 rows: next check)
    for s in (0.0625, 0.0, -1.0, under, -under, 1e-40):
        assert _call(dsa, name, s) == dsa.DSA_ERR_WORKSPACE, s


def test_group_calls_refuse_them_too(dsa):
    one = (ctypes.c_void_p * 1)(4096)
    p = ctypes.cast(one, dsa._PP)
    b = ctypes.byref(dsa._Batch(1, 4, 4, 256, FAKE, FAKE, FAKE))
    for dt, scale, want in ((2, 2.0 ** 87, dsa.DSA_ERR_UNSUPPORTED), (2, 0.0625, dsa.DSA_ERR_WORKSPACE),
                            (0, 2.0 ** 87, dsa.DSA_ERR_WORKSPACE)):
        g = dsa._Group(b"F", 16, 64, scale, dsa.DSA_BF16, 100, 100, p, p, p, p, None, p, None, p, p, None, dt)
        assert dsa.lib.indexshare_group_forward(ctypes.byref(g), b, FAKE, FAKE, 128, None) == want, (dt, scale)
