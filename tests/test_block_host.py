"""CPU checks of the host side of the microscaled 4-bit operators and layer norm."""
import pytest

import bit_quantized_tensor_gb300 as qg

P = 0x10000  # a 256-byte aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return qg.lib()


# ------------------------------------------------------------- addresses

def test_misaligned_statistics_are_refused(L):
    """fp32 vectors at addresses that are no multiple of 4 (a kernel would fault on them)."""
    for mean, rstd in ((P + 2, P), (P, P + 1)):
        assert L.layer_norm(1, 4, 64, P, 64, None, None, 1, 1e-5, P, 64, mean, rstd, None) == 3
        assert L.layer_norm_fp4(0, 1, 4, 64, P, 64, None, None, 1, 1e-5, None, P, P, mean, rstd, None) == 3
    for bad in range(4):
        v = [P + 2 if i == bad else P for i in range(4)]
        assert L.layer_norm_backward(1, 4, 64, P, 64, P, 64, None, 1, v[0], v[1], P, 64, v[2], v[3], P, BIG, None) == 3


# ------------------------------------------------------------- what the norm's bulk copies fetch

ROW_PIECES = r"""
#include <cstdio>
#include <initializer_list>
#include "row_pieces.h"
using namespace qg;
// Every matrix of short rows at every place: what is fetched for a row lies in the
// matrix, in whole pieces, and with what is copied by hand it is the row.
int main() {
    long n = 0;
    for (int elem : {2, 4})
        for (int off = 0; off < 32; off += elem)
            for (int D = 1; D <= 40; ++D)
                for (int gap : {0, 1, 2, 3, 7, 8, 11})
                    for (int M : {1, 2, 3, 7, 8, 9, 17, 40}) {
                        const uintptr_t start = 4096 + off, rb = D * elem, ld = (D + gap) * elem;
                        const uintptr_t stop = start + (M - 1) * ld + rb;
                        const RowBounds m = row_bounds(reinterpret_cast<const void*>(start), M, ld, rb);
                        for (int i = 0; i < M; ++i, ++n) {
                            const uintptr_t r = start + i * ld;
                            const RowPieces q = row_pieces(r, rb, m, m.at_end(i));
                            const uintptr_t b = q.a + q.bytes;
                            bool ok = q.start == r && q.end == r + rb && q.base <= r && r - q.base < 16;
                            ok = ok && (!q.bytes || (q.a % 16 == 0 && q.bytes % 16 == 0 && q.a >= start && b <= stop));
                            ok = ok && (!q.bytes || q.a >= q.base);  // inside the slot, whose end is 31 bytes on
                            ok = ok && (!q.bytes || b <= ((q.end + 15) & ~uintptr_t(15)));
                            // [start, head_end), [a, b), [tail, end) follow one another without a gap
                            ok = ok && q.head_end() <= q.end && q.tail() <= q.end + 15;
                            if (q.bytes)
                                ok = ok && q.a <= (q.start > q.head_end() ? q.start : q.head_end()) && q.tail() == b;
                            else
                                ok = ok && q.head_end() == q.end && q.tail() == q.end;
                            // 32 lanes of 2 bytes copy each by hand; only rows at an end have any
                            const uintptr_t head = q.head_end() > q.start ? q.head_end() - q.start : 0;
                            const uintptr_t tail = q.end > q.tail() ? q.end - q.tail() : 0;
                            ok = ok && head <= 64 && tail <= 64 && (m.at_end(i) || (!head && !tail && q.bytes));
                            if (!ok) {
                                std::printf("elem %d offset %d D %d gap %d M %d row %d\n", elem, off, D, gap, M, i);
                                return 1;
                            }
                        }
                    }
    std::printf("%ld rows\n", n);
    return 0;
}
"""


def test_bulk_copies_stay_inside_the_matrix(tmp_path):
    import shutil
    import subprocess

    from bit_quantized_tensor_gb300 import _build
    src, exe = tmp_path / "row_pieces.cpp", tmp_path / "row_pieces"
    src.write_text(ROW_PIECES)
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", _build.CSRC, str(src),
                    "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


# ------------------------------------------------------------- streams and devices
#
# The calls on stand-ins for torch and for the library: which stream an allocation is
# made on and a kernel is launched on, and that nothing is launched when refused.

class Stream:
    def __init__(self, handle, index=0):
        self.cuda_stream, self.device = handle, Device(index)


class Device:
    def __init__(self, index):
        self.index = index

    def __eq__(self, other):
        return self.index == other.index

    def __str__(self):
        return f"cuda:{self.index}"


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.device = tuple(shape), dtype, Device(index)

    def stride(self):
        return tuple(self.numel() // max(1, self._upto(i + 1)) for i in range(len(self.shape)))

    def _upto(self, n):
        k = 1
        for s in self.shape[:n]:
            k *= s
        return k

    def numel(self):
        return self._upto(len(self.shape))

    def element_size(self):
        return 4

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


class Torch:
    """What the host side uses of torch, with a current stream and a log of allocations."""

    def __init__(self):
        import torch
        self.uint8, self.float32, self.bfloat16, self.float16 = torch.uint8, torch.float32, torch.bfloat16, torch.float16
        self.Tensor, self.current, self.allocated_on = Tensor, Stream(1), []
        self.cuda, self._C = self, self

    def empty(self, shape, dtype, device):
        self.allocated_on.append(self.current.cuda_stream)
        return Tensor(shape if isinstance(shape, tuple) else (shape,), dtype, device.index)

    def current_device(self):
        return self.current.device.index

    def _cuda_getCurrentRawStream(self, index):
        return self.current.cuda_stream

    def stream(self, s):
        import contextlib

        @contextlib.contextmanager
        def swap():
            before, self.current = self.current, s
            yield
            self.current = before
        return swap()


class Library:
    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        def call(*args):
            if name == "qg_workspace_size":
                return 4096
            self.launched.append((name, args[-1]))
            return 0
        return call


class Nothing:
    def __getattr__(self, name):
        return lambda *args: None


@pytest.fixture
def stand_ins(monkeypatch):
    torch, lib = Torch(), Library()
    monkeypatch.setattr(qg, "_torch_module", torch)
    monkeypatch.setattr(qg, "lib", lambda: lib)
    monkeypatch.setattr(qg, "_ordinary", Nothing)
    monkeypatch.setattr(qg, "_dtype_ids", None)
    return torch, lib


def calls(torch, index=0):
    """Every call, 64 tokens of 64 values by 64 outputs, operands on cuda:index."""
    x = Tensor((64, 64), torch.bfloat16, index)
    q, s = Tensor((64, 32), torch.uint8, index), Tensor((1, 1, 512), torch.uint8, index)
    v = Tensor((64,), torch.float32, index)
    return {
        "fp4_tensor_scale": lambda **kw: qg.fp4_tensor_scale(x, **kw),
        "fp4_quantize": lambda **kw: qg.fp4_quantize(x, **kw),
        "fp4_quantize_both": lambda **kw: qg.fp4_quantize_both(x, **kw),
        "fp4_dequantize": lambda **kw: qg.fp4_dequantize(q, s, 64, **kw),
        "fp4_gemm": lambda **kw: qg.fp4_gemm(q, s, q, s, 64, **kw),
        "fp4_linear": lambda **kw: qg.fp4_linear(x, q, s, **kw),
        "fp4_linear_backward": lambda **kw: qg.fp4_linear_backward(x, x, q, s, **kw),
        "layer_norm": lambda **kw: qg.layer_norm(x, **kw),
        "layer_norm_fp4": lambda **kw: qg.layer_norm_fp4(x, stats=True, **kw),
        "layer_norm_backward": lambda **kw: qg.layer_norm_backward(x, x, None, v, v, **kw),
    }


CALLS = list(calls(Torch()))


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_allocates_belongs_to_its_stream(stand_ins, name):
    torch, lib = stand_ins
    calls(torch)[name]()
    assert lib.launched == [(name, 1)] and set(torch.allocated_on) == {1}
    lib.launched.clear(), torch.allocated_on.clear()
    calls(torch)[name](stream=Stream(2))
    assert lib.launched == [(name, 2)] and set(torch.allocated_on) == {2}
    assert torch.current.cuda_stream == 1


@pytest.mark.parametrize("name", CALLS)
def test_operands_on_another_device_are_refused(stand_ins, name):
    """A launch goes to the current device, which cannot be relied on to reach another's memory."""
    torch, lib = stand_ins
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        calls(torch, index=1)[name]()
    with pytest.raises(ValueError, match="is on cuda:0, the current device is cuda:1"):
        calls(torch)[name](stream=Stream(2, index=1))
    assert not lib.launched
    calls(torch, index=1)[name](stream=Stream(2, index=1))  # which makes cuda:1 the current one
    assert lib.launched == [(name, 2)]


# ------------------------------------------------------------- workspaces

def test_workspace_of_the_norms_gradient(L):
    """The rows of partial sums that a launch can leave: one an SM, fewer for long rows."""
    for D, parts in ((1, 160), (8192, 160), (8193, 40), (16384, 40)):
        assert L.qg_workspace_size(qg.QG_OP_LAYER_NORM_BACKWARD, 1, 1, D) == parts * 2 * D * 4
