"""Refusals of the served-layer calls (delta rule, key-value cache) that need no GPU: bad handles, geometries and
arguments are errors before any CUDA call, and the binding checks shapes and strides."""
import ctypes

import pytest

from quantized_recurrent_state_b200 import build as qbuild
from quantized_recurrent_state_b200 import stepq

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return stepq.lib()


def _einval(rc, part):
    assert rc == stepq.EINVAL
    assert part in stepq.lib().stepq_last_error().decode()


def test_delta_calls_refuse_null_handles(lib):
    t = stepq.Tokens(dtype=stepq.BF16, n_qk_heads=1)
    _einval(lib.stepq_delta_step(None, 0, None, None, 1, 1, ctypes.byref(t)), "null context")
    _einval(lib.stepq_delta_step(None, 0, None, None, 1, 0, ctypes.byref(t)), "n_tok 0")
    _einval(lib.stepq_delta_prefill(None, 0, None, None, None, 1, None, 1, ctypes.byref(t)), "null context")
    _einval(lib.stepq_ctx_wait_stream(None, None), "null context")
    _einval(lib.stepq_stream_wait_ctx(None, None), "null context")


@pytest.mark.parametrize("args, part", [
    ((6, 8, 128, 16, 4), "width 6"), ((8, 0, 128, 16, 4), "n_heads 0"), ((8, 5000, 128, 16, 4), "n_heads 5000"),
    ((8, 8, 96, 16, 4), "d 96"), ((8, 8, 128, 24, 4), "page_tokens 24"), ((8, 8, 128, 0, 4), "page_tokens 0"),
    ((8, 8, 128, 1 << 17, 4), "page_tokens 131072"), ((8, 8, 128, 16, 0), "n_pages 0")])
def test_kv_create_refuses_geometries(lib, args, part):
    h = ctypes.c_void_p()
    _einval(lib.stepq_kv_create(*args, ctypes.byref(h)), part)
    assert not h.value


def test_kv_calls_refuse_null_handles(lib):
    _einval(lib.stepq_kv_create(8, 1, 128, 16, 1, None), "null argument")
    _einval(lib.stepq_kv_append(None, None, 0, 1, None, None, 0, 0, None, None), "null cache handle")
    _einval(lib.stepq_kv_read(None, None, 1, None, 1, None, None, 1, 0, None, None, 0, 0, None), "null cache handle")
    _einval(lib.stepq_kv_attend(None, None, 1, None, 1, None, 0, 1, 1, None, 0, 1.0, None, 0, None, None, None),
            "null cache handle")
    _einval(lib.stepq_kv_check(None, None), "null cache handle")
    assert lib.stepq_kv_bytes(None) == 0
    assert lib.stepq_kv_attend_workspace_bytes(None, 1, 1, 1, 1) == 0
    lib.stepq_kv_free(None)


def test_kv_wait_limit_refuses_a_null_handle(lib):
    _einval(lib.stepq_kv_set_wait_limit(None, 0, 0), "null cache handle")


def test_row_stride():
    x = torch.zeros(6, 10, 16)
    assert stepq._row_stride(x[:, 2:5], (6,), 3, 16, "x") == 160
    assert stepq._row_stride(x[:1, 2:5], (1,), 3, 16, "x") == 48          # a single row: any stride will do
    assert stepq._row_stride(x.view(2, 3, 10, 16)[:, :, 1:3], (2, 3), 2, 16, "x") == 160
    assert stepq._row_stride(x.view(6, 1, 10, 16), (6, 1), 10, 16, "x") == 160
    assert stepq._row_stride(x.view(1, 6, 10, 16), (1, 6), 10, 16, "x") == 160
    for bad, lead, heads in [(x[:, ::2], (6,), 5), (x.transpose(1, 2), (6,), 16), (x.view(2, 3, 10, 16)[:, :2], (2, 2), 10),
                             (x, (6,), 9), (x, (5,), 10)]:
        with pytest.raises(stepq.StepqError) as e:
            stepq._row_stride(bad, lead, heads, bad.shape[-1], "x")
        assert e.value.code == stepq.EINVAL


def test_host_tensors_are_refused():
    with pytest.raises(stepq.StepqError, match="is on cpu"):
        stepq._rows(torch.zeros(2, 1, 16), 0, torch.float32, (2,), 1, 16, "q")
    with pytest.raises(stepq.StepqError, match="is on cpu"):
        stepq._dense(torch.zeros(2), 0, torch.float32, 2, "beta")
