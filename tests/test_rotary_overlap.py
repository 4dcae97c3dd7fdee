"""Rotations whose buffers are the same memory: each output element would be
written while others are still to be read from it, so they are refused."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from lora_linear_fine_b200 import build
    build.build(quiet=True)
    import lora_linear_fine_b200 as L
    return L


def test_c_entry_point(lib):
    def f(Q=1 << 20, K=2 << 20, Yq=3 << 20, Yk=4 << 20, M=4, kv=2):
        return lib.lora_linear_rotary(lib.make_rotary_desc(M, 2, kv, 64, 32), lib.make_rope_desc(16, 16, 16, 8, 64),
                                      Q, K, Yq, Yk, 16, 256, None)
    a, b, c = 1 << 20, 2 << 20, 3 << 20
    assert f(Yq=a, Yk=a, K=a) == 1              # in place, one tensor for q and k
    assert f(Yk=c) == 1                         # two outputs in one place
    assert f(Yq=b) == 1 and f(Yk=a) == 1        # an output over the other's input
    assert f() not in (1, 2, 3, 5)
    assert f(K=a) not in (1, 2, 3, 5)           # one input turned twice, to two places
    assert f(Yq=a, Yk=b) not in (1, 2, 3, 5)    # in place
    assert f(M=0, Q=None, K=None, Yq=None, Yk=None) not in (1, 2, 3, 5)
    assert f(kv=0, K=None, Yk=None) not in (1, 2, 3, 5)


@pytest.mark.parametrize("first,rows", [(0, 4), (3, 4), (0, 3)])
def test_in_place_over_one_tensor(lib, first, rows):
    import torch
    X = torch.zeros(8, 128, dtype=torch.bfloat16)
    pos, table = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 16)
    K = X[first:first + 4] if rows == 4 else X.flatten()[64:64 + 4 * 64].view(4, 64)
    with pytest.raises(lib.LoraError, match="overlap"):
        lib.rotary(X[:4], K, pos, table, table, 64, inplace=True)


def test_in_place_beside_each_other(lib):
    """Not refused for that: these lie on the CPU, which is the next thing to be seen."""
    import torch
    X = torch.zeros(8, 128, dtype=torch.bfloat16)
    pos, table = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 16)
    with pytest.raises(lib.LoraError, match="CUDA"):
        lib.rotary(X[:4], X[4:], pos, table, table, 64, inplace=True)
