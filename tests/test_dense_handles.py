"""Handles over 8-bit rows, without a GPU: the tensors here say that they are on one, and the library is one that only
records its calls."""
import struct

import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import dense as D


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def on_gpu(t):
    return t.as_subclass(OnGpu)


def zeros(*shape, dtype=torch.uint8):
    return on_gpu(torch.zeros(shape, dtype=dtype))


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(D, "_LIB", lib)
    monkeypatch.setattr(D, "_stream", lambda stream, device: 0)
    return lib


def handle(rows=6, k=64):
    return D.Fp8Rows(zeros(rows, k), zeros(rows, 4))


def calls_with(r):
    """A call of each entry point with r in each of its places."""
    x, y = zeros(6, 64, dtype=torch.bfloat16), zeros(6, 6, dtype=torch.bfloat16)
    other, ws = handle(), zeros(4096)
    return [lambda: D.moe_fp8_quantize_rows(x, r), lambda: D.moe_fp8_gemm(r, other, y), lambda: D.moe_fp8_gemm(other, r, y),
            lambda: D.moe_fp8_linear(x, r, y, ws), lambda: D.moe_residual_norm(x, quantized=r)]


def test_handles_reach_the_library_as_they_are(lib):
    r = handle()
    for call in calls_with(r):
        call()
    assert [name for name, _ in lib.calls] == ["moe_fp8_quantize_rows", "moe_fp8_gemm", "moe_fp8_gemm", "moe_fp8_linear", "moe_residual_norm"]
    want = struct.pack("PPqq", r.codes.data_ptr(), r.scales.data_ptr(), 64, 4)
    assert lib.calls[0][1][5] == want and lib.calls[1][1][0] == want and lib.calls[2][1][2] == want and lib.calls[3][1][5] == want
    assert lib.calls[4][1][0].endswith(want)


CHANGES = {
    "codes are others": lambda r: setattr(r, "codes", zeros(6, 64)),
    "scales are others": lambda r: setattr(r, "scales", zeros(6, 4)),
    "codes' data": lambda r: setattr(r.codes, "data", zeros(6, 64)),
    "scales' data": lambda r: setattr(r.scales, "data", zeros(6, 4)),
    "codes set": lambda r: r.codes.set_(zeros(6, 64)),
    "codes larger": lambda r: r.codes.resize_(600, 64),
    "storage gone": lambda r: r.codes.untyped_storage().resize_(0),
}


@pytest.mark.parametrize("change", CHANGES)
def test_handles_whose_tensors_changed_are_refused(lib, change):
    """Calls would go on with the old address, whose memory may be someone else's by then."""
    r = handle()
    calls, keep = calls_with(r), [r.codes, r.scales]
    CHANGES[change](r)
    for call in calls:
        with pytest.raises(ValueError, match="its tensors"):
            call()
    assert not lib.calls and keep


def test_values_written_in_place_are_no_change(lib):
    r = handle()
    r.codes.fill_(7)
    r.scales.copy_(zeros(6, 4))
    for call in calls_with(r):
        call()
    assert len(lib.calls) == 5


def test_memory_that_a_handle_was_made_of_stays(lib):
    """A tensor that lets go of its memory and gets other memory at the same address would look unchanged."""
    codes = zeros(6, 64)
    r, storage = D.Fp8Rows(codes, zeros(6, 4)), codes.untyped_storage()._cdata
    codes.data = zeros(6, 64)
    assert any(t.untyped_storage()._cdata == storage for t in r.held)


@pytest.mark.parametrize("what", [torch.zeros((6, 64), dtype=torch.uint8), "rows"])
def test_other_things_than_handles_are_refused(lib, what):
    for call in calls_with(what):
        with pytest.raises(ValueError, match="must be Fp8Rows"):
            call()
    assert not lib.calls


@pytest.mark.parametrize("n", [-1, 7, 100])
def test_a_handle_over_more_rows_than_there_are(n):
    with pytest.raises(ValueError, match="6 rows"):
        handle().rows(n)


def test_a_handle_over_the_first_rows():
    r = handle()
    assert r.rows(6) is r and r.rows(2).n == 2 and r.rows(0).n == 0 and r.rows(2).at == r.at


@pytest.mark.parametrize("tokens,k", [(2 ** 32 + 1, 64), (1, 2 ** 32 + 64), (-2 ** 32 + 1, 64), (2 ** 31, 64), (-1, 64), (4, 40)])
def test_workspaces_of_sizes_that_an_int_does_not_hold(native, tokens, k):
    """Their low 32 bits would be another size."""
    with pytest.raises(ValueError, match="no product of"):
        D.linear_workspace(tokens, k, "cpu")


def test_a_workspaces_size(native):
    assert D.linear_workspace(5, 64, "cpu").numel() == D.load().moe_fp8_linear_workspace_size(5, 64) > 0
