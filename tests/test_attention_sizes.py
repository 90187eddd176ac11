"""CPU checks of the attention layer's operators: workspace sizes, a refusal, the kernels' table."""
import pytest

import bit_quantized_tensor_gb300 as qg


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return qg.lib()


@pytest.mark.parametrize("N,K", [(4096, 4096), (11008, 4096), (1001, 2304), (8192, 8192), (17, 20000), (4096, 130000), (64, 1)])
def test_a_workspace_for_many_tokens_serves_fewer(L, N, K):
    sizes = [L.qg_workspace_size(qg.QG_OP_S8_LINEAR, m, N, K) for m in list(range(1, 4400)) + [5000, 8192, 1 << 20]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_scales_that_leave_fp32_in_powers_of_two_are_refused(L, scale):
    p = 0x10000
    assert L.kv8_attention(1, 2, 4, 4, 2, 64, p, 256, p, p, p, p, 8, 16, p, 4, p, p, scale, 1, p, 256, p, 1 << 40,
                           None) == 1
    assert L.kv8_attention(1, 0, 4, 4, 2, 64, p, 256, p, p, p, p, 8, 16, p, 4, p, p, 2e38, 1, p, 256, p, 1 << 40,
                           None) == 0


def test_tensor_core_kernels_are_in_the_table(L):
    names = [r["kernel"] for r in qg.kernel_budgets(table="block")]
    for tile in (32, 64, 128):
        assert f"s8_gemm_kernel<{tile}>" in names
    for dtype in ("f16", "bf16"):
        for D in (64, 128):
            assert all(f"k_kv8_attention_rows<{dtype},{D},{form}>" in names for form in ("whole", "some", "split"))
            assert f"k_kv8_attention_rows_join<{dtype},{D}>" in names
