"""The entry points around 8-bit experts without a GPU: sizes, and what they refuse before
launching."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._load_builder().build()
    import combine_fp32_router_gb300 as moe
    return moe


FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD1 = ctypes.c_void_p((1 << 20) + 1)
BIG = 1 << 31


def caller(f, ok):
    def with_(changes):
        a = list(ok)
        for i, v in changes.items():
            a[i] = v
        return f(*a)
    return with_


def refused(lib, with_, invalid=(), unsupported=()):
    for c in invalid:
        assert with_(c) == lib.MOE_ERR_INVALID_ARG, c
    for c in unsupported:
        assert with_(c) == lib.MOE_ERR_UNSUPPORTED, c


def test_sizes(lib):
    raw = lib.library()
    for c in (0, 1, 128, 129, 7168):
        assert lib.moe_fp8_row_bytes(c) == raw.moe_fp8_row_bytes(c) == -(-c // 128) * 128
    assert raw.moe_fp8_row_bytes(-1) == 0
    assert lib.moe_sort_rows_bound(0, 2, 8) == 0
    assert lib.moe_sort_rows_bound(1, 2, 8) == 256
    assert lib.moe_sort_rows_bound(16384, 8, 256) == -(-(16384 * 8 + 127 * 256) // 128) * 128
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 2, 0), (4, 17, 32), (4, 2, 1025), (1 << 30, 2, 8)):
        assert lib.moe_sort_rows_bound(*bad) == 0
        assert lib.moe_sort_workspace_bytes(bad[0], bad[2], bad[1]) == 0
    assert 0 < lib.moe_sort_workspace_bytes(64, 8, 2) < lib.moe_sort_workspace_bytes(65536, 8, 2)
    assert lib.moe_rmsnorm_workspace_bytes(1000, 7168) >= 7168 * 4
    for bad in ((-1, 128), (4, 0), (4, 16385), (BIG, 128)):
        assert lib.moe_rmsnorm_workspace_bytes(*bad) == 0


def test_quantize_refusals(lib):
    raw = lib.library()
    with_ = caller(raw.moe_quantize_rows_fp8, (FAKE, 0, 4, 64, 64, 0, None, FAKE, FAKE, None))
    refused(lib, with_,
            invalid=[{0: None}, {1: 3}, {1: -1}, {2: -1}, {3: 0}, {4: 63}, {4: -1}, {5: 2}, {5: 1}, {6: ODD1}, {7: None},
                     {7: ODD}, {8: None}, {8: ODD1}, {0: ODD1}, {5: 1, 4: 127}],
            unsupported=[{2: 1 << 32}, {3: (1 << 20) + 1, 4: 1 << 21}])
    assert with_({2: 0}) == lib.MOE_OK
    with_ = caller(raw.moe_dequantize_rows_fp8, (FAKE, FAKE, 4, 64, 0, FAKE, None))
    refused(lib, with_, invalid=[{0: None}, {1: None}, {5: None}, {5: ODD}, {0: ODD}, {1: ODD1}, {2: -1}, {3: 0}, {4: 3}],
            unsupported=[{2: BIG}, {3: (1 << 20) + 1}])
    assert with_({2: 0}) == lib.MOE_OK
    with_ = caller(raw.moe_quantize_blocks_fp8, (FAKE, 2, 64, 64, 1, FAKE, FAKE, None))
    refused(lib, with_, invalid=[{0: None}, {0: ODD}, {1: 0}, {2: 0}, {3: 0}, {4: 2}, {5: None}, {5: ODD}, {6: ODD1}],
            unsupported=[{1: 1025}, {2: (1 << 20) + 1}, {3: (1 << 20) + 1}])


def test_gemm_refusals(lib):
    with_ = caller(lib.library().moe_gemm_fp8, (FAKE, FAKE, 4, FAKE, FAKE, FAKE, 2, 64, 64, FAKE, 0, None))
    refused(lib, with_,
            invalid=[{0: None}, {1: None}, {4: None}, {5: None}, {9: None}, {0: ODD}, {4: ODD}, {1: ODD1}, {5: ODD1},
                     {9: ODD1}, {2: -1}, {3: None}, {3: ODD1}, {6: 0}, {7: 0}, {8: 0}, {10: lib.MOE_DTYPE_F16}, {10: 9}],
            unsupported=[{2: BIG}, {6: 1025}, {7: (1 << 20) + 1}, {8: (1 << 20) + 1}])
    assert with_({2: 0}) == lib.MOE_OK


def test_norm_refusals(lib):
    raw = lib.library()
    ok = (FAKE, 64, FAKE, FAKE, 0, 0, 4, 64, 1e-6, FAKE, FAKE, FAKE, FAKE, FAKE, None)
    refused(lib, caller(raw.moe_rmsnorm, ok),
            invalid=[{0: None}, {1: 63}, {1: -1}, {2: None}, {3: None}, {4: 3}, {5: 1}, {6: -1}, {7: 0}, {8: -1.0},
                     {8: float("nan")}, {9: None}, {10: None, 11: None, 12: None}, {11: None}, {12: None}, {11: ODD},
                     {0: ODD1}, {2: ODD1}, {3: ODD1}, {9: ODD1}, {10: ODD1}, {12: ODD1}, {13: ODD1}],
            unsupported=[{6: BIG}, {7: 16385, 1: 16385}])
    assert caller(raw.moe_rmsnorm, ok)({6: 0}) == lib.MOE_OK
    need = lib.moe_rmsnorm_workspace_bytes(4, 64)
    ok = (FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 4, 64, FAKE, FAKE, FAKE, need, None)
    with_ = caller(raw.moe_rmsnorm_backward, ok)
    refused(lib, with_,
            invalid=[{i: None} for i in (0, 1, 2, 3, 9, 11)] + [{i: ODD1} for i in (0, 1, 2, 3, 4, 9, 10, 11)] +
            [{5: 3}, {6: 1}, {7: -1}, {8: 0}, {11: ODD}],
            unsupported=[{7: BIG}, {8: 16385}])
    assert with_({12: need - 1}) == lib.MOE_ERR_WORKSPACE
    assert with_({7: 0, 10: None, 11: None}) == lib.MOE_OK


def test_sort_refusals(lib):
    raw = lib.library()
    need, n = lib.moe_sort_workspace_bytes(64, 8, 2), lib.moe_sort_rows_bound(64, 2, 8)
    ok = (FAKE, 64, FAKE, 2, FAKE, 64, 2, 8, FAKE, n, FAKE, FAKE, FAKE, FAKE, FAKE, need, None)
    with_ = caller(raw.moe_sort_tokens, ok)
    refused(lib, with_,
            invalid=[{i: None} for i in (0, 2, 4, 8, 10, 11, 12, 13, 14)] + [{i: ODD1} for i in (2, 4, 10, 11, 12, 13, 14)] +
            [{1: 0}, {3: -1}, {3: 0}, {5: -1}, {6: 0}, {7: 0}, {9: n - 1}, {9: BIG}, {14: ODD}],
            unsupported=[{6: 17}, {7: 1025}, {5: 1 << 30}, {1: (1 << 20) + 1}, {3: (1 << 20) + 1}])
    assert with_({15: need - 1}) == lib.MOE_ERR_WORKSPACE
    ok = (FAKE, 0, 100, FAKE, FAKE, 64, 2, 32, FAKE, FAKE, None)
    with_ = caller(raw.moe_unsort_tokens, ok)
    refused(lib, with_,
            invalid=[{i: None} for i in (0, 4, 8, 9)] + [{i: ODD1} for i in (0, 3, 4, 8, 9)] +
            [{1: 3}, {2: -1}, {5: -1}, {6: 0}, {7: 0}, {9: ODD}],
            unsupported=[{2: BIG}, {5: 1 << 31}, {6: 17}, {7: 65537}])
    assert with_({5: 0}) == lib.MOE_OK
    ok = (FAKE, 0, 100, FAKE, 64, 2, 32, FAKE, FAKE, None)
    refused(lib, caller(raw.moe_sort_tokens_backward, ok), invalid=[{0: None}, {3: None}, {7: None}, {8: None}, {1: 7}])
    ok = (FAKE, FAKE, 0, 100, FAKE, FAKE, 64, 2, 32, FAKE, FAKE, FAKE, None)
    with_ = caller(raw.moe_unsort_tokens_backward, ok)
    refused(lib, with_,
            invalid=[{i: None} for i in (0, 1, 4, 5, 9, 11)] + [{i: ODD1} for i in (0, 1, 4, 5, 9, 10, 11)] +
            [{2: 3}, {3: -1}, {6: -1}, {7: 0}, {8: 0}],
            unsupported=[{3: BIG}, {6: 1 << 31}, {7: 17}, {8: 65537}])
    assert with_({6: 0}) == lib.MOE_OK


def test_wrappers_refuse_host_tensors_and_wrong_shapes(lib):
    f32, u8, i32, bf = torch.float32, torch.uint8, torch.int32, torch.bfloat16
    z = lambda *s, dt=f32: torch.zeros(*s, dtype=dt)
    x = z(4, 64, dt=bf)
    calls = [
        lambda: lib.moe_quantize_rows_fp8(x),
        lambda: lib.moe_quantize_rows_fp8(z(4, 63, dt=bf), swiglu=True),
        lambda: lib.moe_quantize_rows_fp8(x.t()),
        lambda: lib.moe_quantize_rows_fp8(z(4, 64, dt=torch.float64)),
        lambda: lib.moe_quantize_rows_fp8(z(4)),
        lambda: lib.moe_dequantize_rows_fp8(z(4, 128, dt=u8), z(4, 1), 64),
        lambda: lib.moe_dequantize_rows_fp8(z(4, 128, dt=u8), z(4, 1), 129),
        lambda: lib.moe_dequantize_rows_fp8(z(4, 128, dt=u8), z(4, 1), 0),
        lambda: lib.moe_quantize_blocks_fp8(z(1, 64, 64, dt=bf)),
        lambda: lib.moe_quantize_blocks_fp8(z(1, 64, 64)),
        lambda: lib.moe_gemm_fp8(z(4, 128, dt=u8), z(4, 1), z(8, 128, dt=u8), z(1, 1), z(4, 8), 100),
        lambda: lib.moe_gemm_fp8(z(4, 128, dt=u8), z(4, 1), z(8, 128, dt=u8), z(1, 1), z(4, 9), 100),
        lambda: lib.moe_gemm_fp8(z(3, 128, dt=u8), z(3, 1), z(8, 128, dt=u8), z(1, 1), z(4, 8), 100),
        lambda: lib.moe_rmsnorm(x, z(64), 1e-6, out=x),
        lambda: lib.moe_rmsnorm(z(4), z(64), 1e-6, out=x),
        lambda: lib.moe_rmsnorm_backward(x, x, z(64), z(4), x, z(64), z(256, dt=u8)),
        lambda: lib.moe_sort_tokens(x, z(4, 2, dt=i32), z(512, 64, dt=bf), z(8, dt=i32), z(512, dt=i32), z(4, 2, dt=i32),
                                    z(256, dt=u8)),
        lambda: lib.moe_sort_tokens(x, z(5, 2, dt=i32), z(512, 64, dt=bf), z(8, dt=i32), z(512, dt=i32), z(5, 2, dt=i32),
                                    z(256, dt=u8)),
        lambda: lib.moe_sort_tokens_backward(x, z(2, 2, dt=i32), x, z(16, dt=u8)),
        lambda: lib.moe_unsort_tokens(x, z(2, 2), z(2, 2, dt=i32), z(2, 64, dt=bf), z(16, dt=u8)),
        lambda: lib.moe_unsort_tokens_backward(z(2, 64, dt=bf), x, z(2, 2), z(2, 2, dt=i32), x, z(2, 2), z(16, dt=u8)),
    ]
    for i, c in enumerate(calls):
        with pytest.raises(ValueError):
            c()
            pytest.fail("call %d was accepted" % i)
