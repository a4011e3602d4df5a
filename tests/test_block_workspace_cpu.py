"""A workspace made for the largest batch serves every smaller one: the sizes
never fall as rows are added."""

import ctypes

import pytest

OK = 0


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_fp32_gb300 import build
    build.build()
    import mixture_experts_layer_fp32_gb300 as m
    return m


def _grows(sizes):
    return all(b >= a for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("N,K", [(14336, 7168), (14336, 4096), (32000, 4096), (128256, 4096),
                                 (4096, 14336), (1000, 65536), (64, 32), (333, 96)])
def test_linear(moe, N, K):
    size = ctypes.c_size_t()

    def ask(rows):
        assert moe.lib().moe_workspace_size_linear_w4(rows, N, K, ctypes.byref(size)) == OK
        return size.value

    rows = list(range(0, 70)) + [127, 128, 129, 192, 193, 256, 257, 384, 385, 449, 512, 513, 577,
                                 640, 705, 769, 896, 897, 1023, 1024, 1025, 4096]
    sizes = [ask(r) for r in rows]
    assert _grows(sizes)


@pytest.mark.parametrize("h,E,k,f", [(4096, 8, 2, 14336), (7168, 256, 8, 2048),
                                     (4096, 128, 8, 1536), (256, 1, 1, 128), (512, 3, 2, 640)])
def test_experts_and_forward(moe, h, E, k, f):
    for ask in (moe.workspace_size_experts_w4, moe.workspace_size_w4):
        sizes = [ask(moe.config(T=T, h=h, E=E, k=k, f=f))
                 for T in list(range(0, 100)) + [128, 256, 511, 512, 513, 1024, 1025]]
        assert _grows(sizes)


@pytest.mark.parametrize("H", [1, 64, 256, 511, 1021, 1023, 1024, 2048, 4096, 4099, 8200, 16384,
                               33000])
def test_norm_backward(moe, H):
    sizes = [moe.workspace_size_norm_backward(rows, H) for rows in range(0, 5000)]
    assert _grows(sizes)
