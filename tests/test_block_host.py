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
