"""The counts behind the error bounds: that they are those of the kernels' plan, without a GPU."""
import pytest

import _sandwich_chain as chain


@pytest.fixture(scope="module")
def rm():
    from rmsnorm_modulate_gb300 import _build

    _build.build()
    import rmsnorm_modulate_gb300 as rm

    return rm


def test_items_are_those_of_the_workspace(rm):
    f = rm.library().sandwich_rmsnorm_modulate_backward_workspace_bytes
    for D in (8, 256, 264, 512, 520, 768, 1024, 2560, 4096, 4104, 6144, 8192, 8200, 12288, 16384):
        for S in (1, 2, 7, 8, 9, 77, 400, 1216, 4216, 21000, 40000, 140000):
            for B in (1, 3):
                assert f(B, S, D) == 12 * D * B * chain.items(S, D)[1], (B, S, D)


def test_counts_by_hand():
    # 4096 values: 512 vectors, four a thread, groups of four warps, two groups of eight warps
    assert chain.shape(512, True) == (512, 4, 4, 2) and chain.shape(512, False) == (512, 4, 4, 4)
    # 4216 rows of them: items of 28 rows, 14 to a group
    assert chain.items(4216, 4096) == (28, 151, 2)
    # 14 + 1 + 5 rounds of 32 slices + 32; shared by one batch: 1 + 1 more
    assert chain.column_additions(1, 4216, 4096, False) == 14 + 1 + 5 + 32
    assert chain.column_additions(1, 4216, 4096, True) == 14 + 1 + 5 + 32 + 2
    # single rows: one item of one row; 16 batches at a time
    assert chain.column_additions(400, 1, 4096, True) == 1 + 0 + 1 + 4 + 25 + 16
    for Dv in range(1, 2049):
        for backward in (False, True):
            nv, v, warps, groups = chain.shape(Dv, backward)
            assert groups >= 1 and 32 * v * warps >= nv and v <= 4
            assert groups * warps <= (8 if backward and v > 2 else 16)
            if groups > 1 or Dv > 1024:  # the places that a row's parts are joined from
                assert -(-warps // 4) * (2 if Dv > 1024 else 1) <= 6
