"""The 4-bit entry points without a GPU: sizes, and what they refuse before launching."""
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


def test_sizes(lib):
    assert [lib.moe_fp4_row_bytes(c) for c in (1, 128, 129, 7168)] == [64, 64, 128, 3584]
    assert lib.moe_fp4_scale_bytes(1, 1) == 128 * 4
    assert lib.moe_fp4_scale_bytes(129, 129) == 256 * 8
    assert lib.moe_fp4_scale_bytes(0, 128) == 0 and lib.moe_fp4_scale_bytes(-1, 128) == 0
    assert lib.moe_few_workspace_bytes(1, 128, 8, 2, 128) > 0
    for bad in ((33, 128, 8, 2, 128), (1, 100, 8, 2, 128), (1, 128, 8, 2, 130),
                (1, 128, 8, 9, 128), (1, 128, 2048, 2, 128), (1, 128, 32, 17, 128),
                (-1, 128, 8, 2, 128)):
        assert lib.moe_few_workspace_bytes(*bad) == 0


def test_quantize_refusals(lib):
    f = lib.library().moe_quantize_rows_fp4
    ok = (FAKE, 0, 4, 64, 64, FAKE, FAKE, None)

    def with_(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i, v in ((0, None), (1, 3), (1, -1), (2, -1), (3, 0), (3, -5), (4, 63), (4, -1), (5, None),
                 (5, ODD), (6, None), (6, ODD), (0, ctypes.c_void_p((1 << 20) + 1))):
        assert with_(i, v) == lib.MOE_ERR_INVALID_ARG, (i, v)
    assert with_(2, 1 << 32) == lib.MOE_ERR_UNSUPPORTED
    assert f(FAKE, 0, 4, (1 << 20) + 1, 1 << 21, FAKE, FAKE, None) == lib.MOE_ERR_UNSUPPORTED
    assert with_(2, 0) == lib.MOE_OK


def test_dequantize_and_weights_refusals(lib):
    f = lib.library().moe_dequantize_rows_fp4
    assert f(FAKE, FAKE, 1, 4, 64, 5, FAKE, None) == lib.MOE_ERR_INVALID_ARG
    assert f(FAKE, FAKE, 1, 4, 64, 0, ODD, None) == lib.MOE_ERR_INVALID_ARG
    assert f(None, FAKE, 1, 4, 64, 0, FAKE, None) == lib.MOE_ERR_INVALID_ARG
    assert f(FAKE, FAKE, 4, 1 << 30, 64, 0, FAKE, None) == lib.MOE_ERR_UNSUPPORTED
    assert f(FAKE, FAKE, 0, 4, 64, 0, FAKE, None) == lib.MOE_OK
    g = lib.library().moe_quantize_weights_fp4
    assert g(FAKE, 0, 64, 64, FAKE, FAKE, None) == lib.MOE_ERR_INVALID_ARG
    assert g(FAKE, 1, 0, 64, FAKE, FAKE, None) == lib.MOE_ERR_INVALID_ARG
    assert g(FAKE, 1, 64, 64, None, FAKE, None) == lib.MOE_ERR_INVALID_ARG
    assert g(ODD, 1, 64, 64, FAKE, FAKE, None) == lib.MOE_ERR_INVALID_ARG
    assert g(FAKE, 1025, 64, 64, FAKE, FAKE, None) == lib.MOE_ERR_UNSUPPORTED


def test_gemm_refusals(lib):
    f = lib.library().moe_gemm_fp4
    ok = (FAKE, FAKE, 4, FAKE, FAKE, FAKE, 2, 64, 64, FAKE, 0, None)

    def with_(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i in (0, 1, 4, 5, 9):
        assert with_(i, None) == lib.MOE_ERR_INVALID_ARG
        assert with_(i, ODD) == lib.MOE_ERR_INVALID_ARG
    for i, v in ((2, -1), (3, None), (3, ctypes.c_void_p((1 << 20) + 2)), (6, 0), (7, 0), (8, 0),
                 (10, lib.MOE_DTYPE_F16), (10, 9)):
        assert with_(i, v) == lib.MOE_ERR_INVALID_ARG, (i, v)
    for i, v in ((2, 1 << 31), (6, 1025), (7, (1 << 20) + 1), (8, (1 << 20) + 1)):
        assert with_(i, v) == lib.MOE_ERR_UNSUPPORTED, (i, v)
    assert with_(2, 0) == lib.MOE_OK


def test_few_refusals(lib):
    f = lib.library().moe_forward_few_fp4
    need = lib.moe_few_workspace_bytes(4, 128, 8, 2, 128)
    ok = [FAKE] * 9 + [4, 128, 8, 2, 128, FAKE, FAKE, need, None]

    def with_(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 14, 15):
        assert with_(i, None) == lib.MOE_ERR_INVALID_ARG, i
        assert with_(i, ODD) == lib.MOE_ERR_INVALID_ARG, i
    assert with_(2, ODD) == lib.MOE_ERR_INVALID_ARG
    assert with_(15, ctypes.c_void_p((1 << 20) + 16)) == lib.MOE_ERR_INVALID_ARG
    assert with_(16, need - 1) == lib.MOE_ERR_WORKSPACE
    assert with_(12, 9) == lib.MOE_ERR_INVALID_ARG          # k > E
    for i, v in ((9, 33), (10, 192), (11, 1025), (13, 130), (10, 65664)):
        assert with_(i, v) == lib.MOE_ERR_UNSUPPORTED, (i, v)
    assert with_(9, -1) == lib.MOE_ERR_INVALID_ARG
    assert with_(9, 0) == lib.MOE_OK


def test_python_refusals(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        lib.moe_quantize_rows_fp4(x.t())                    # a row's values apart
    with pytest.raises(ValueError):
        lib.moe_quantize_rows_fp4(x.double())
    with pytest.raises(ValueError):
        lib.moe_quantize_rows_fp4(x, q=torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        lib.moe_quantize_weights_fp4(torch.zeros(1, 32, 32))
    q, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lib.moe_dequantize_rows_fp4(q, s, 200)
    out = torch.zeros(4, 4)
    with pytest.raises(ValueError):
        lib.moe_gemm_fp4(q, s, q, s, out, 500)
    with pytest.raises(ValueError):
        lib.moe_gemm_fp4(q, s, q, s[:100], out, 64)
    with pytest.raises(ValueError):
        lib.moe_gemm_fp4(q, s, q, s, out, 64, counts=torch.zeros(2, dtype=torch.int32))
    w = torch.zeros(2, 128, 64, dtype=torch.uint8)
    b = torch.zeros(1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.moe_forward_few_fp4(b, torch.zeros(1, 3), None, w, w, w, s, s, s, 1, b, s)
    with pytest.raises(ValueError):
        lib.moe_forward_few_fp4(b.float(), torch.zeros(1, 2), None, w, w, w, s, s, s, 1, b, s)


@pytest.fixture
def calls(lib, monkeypatch):
    """The library calls that a wrapper makes, none of which runs."""
    made = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0
    monkeypatch.setattr(lib, "_lib", Recorder())
    return made


def test_codes_of_other_dimensions_or_types_are_refused(lib, calls):
    """A row of codes taken for a matrix would have its bytes counted as rows: 3584 of them written
    to an output of one."""
    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8)
    s, out = u8(1 << 18), torch.zeros(64, 4)
    for q in (u8(3584), u8(1, 2, 2, 3584), u8(4, 3584).to(torch.int32), torch.zeros(4, 3584)):
        with pytest.raises(ValueError, match="q must hold uint8 codes"):
            lib.moe_dequantize_rows_fp4(q, s, 7168)
    with pytest.raises(ValueError, match="q must hold uint8 codes"):
        lib.moe_dequantize_rows_fp4(u8(64), u8(512), 128)
    for a in (u8(64), u8(64, 1, 64), u8(64, 64).to(torch.int16)):
        with pytest.raises(ValueError, match="aq must hold uint8 codes"):
            lib.moe_gemm_fp4(a, s, u8(4, 64), s, out, 128)
    for b in (u8(64), u8(2, 2, 4, 64), torch.zeros(4, 64)):
        with pytest.raises(ValueError, match="bq must hold uint8 codes"):
            lib.moe_gemm_fp4(u8(64, 64), s, b, s, out, 128)
    x = torch.zeros(1, 128, dtype=torch.bfloat16)
    w = u8(2, 128, 64)
    for i in range(3):
        ws = [w, w, w]
        ws[i] = w.to(torch.float32)
        with pytest.raises(ValueError, match="a weight must hold uint8 codes"):
            lib.moe_forward_few_fp4(x, torch.zeros(1, 2), None, *ws, s, s, s, 1, x, s)
    assert not calls


@pytest.mark.parametrize("given", [False, True])
def test_host_tensors_are_refused(lib, calls, monkeypatch, given):
    """A host address never reaches a kernel, whichever argument it comes in and whether or not a
    stream is given.  (Here the other arguments are host tensors that pass for device ones.)"""
    class Stream:
        cuda_stream = 0

    class Device(torch.Tensor):
        is_cuda = True
    kw = dict(stream=Stream()) if given else {}
    monkeypatch.setattr(lib, "_raw_stream", lambda stream, t: 0)
    monkeypatch.setattr(lib, "_empty", lambda shape, dtype, device, stream: dev(shape, dtype))

    def dev(shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype).as_subclass(Device)
    bf, f32 = torch.bfloat16, torch.float32
    w, s = ((2, 128, 64), torch.uint8), ((2048,), torch.uint8)
    for f, args in (
            (lambda x, q, s: lib.moe_quantize_rows_fp4(x, q, s, **kw),
             [((4, 128), bf), ((4, 64), torch.uint8), s]),
            (lambda q, s: lib.moe_dequantize_rows_fp4(q, s, 128, **kw), [((4, 64), torch.uint8), s]),
            (lambda W: lib.moe_quantize_weights_fp4(W, **kw), [((2, 32, 32), bf)]),
            (lambda a, sa, b, sb, o, c: lib.moe_gemm_fp4(a, sa, b, sb, o, 128, counts=c, **kw),
             [((4, 64), torch.uint8), s, w, s, ((4, 128), f32), ((2,), torch.int32)]),
            (lambda x, lg, r, a, b, c, sa, sb, sc, o, ws:
             lib.moe_forward_few_fp4(x, lg, r, a, b, c, sa, sb, sc, 1, o, ws, **kw),
             [((1, 128), bf), ((1, 2), f32), ((2, 128), f32), w, w, w, s, s, s, ((1, 128), bf),
              ((1 << 20,), torch.uint8)])):
        f(*(dev(*a) for a in args))
        assert len(calls) == 1          # as it is: accepted
        calls.clear()
        for i in range(len(args)):
            mixed = [torch.zeros(a[0], dtype=a[1]) if j == i else dev(*a) for j, a in enumerate(args)]
            with pytest.raises(ValueError, match="must be CUDA tensors"):
                f(*mixed)
        assert not calls
