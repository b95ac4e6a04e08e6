"""CPU: which kernel the integer GEMM takes, from static shapes (a device of
256 compute units, as without one).  At the shapes of the first two tests, or at
their neighbours that were timed, the named kind took 10 % less time than the
next or better."""
import pytest

INT8 = 32


def _mx():
    from block_scaled_precision_03_amd import mxgemm
    return mxgemm


@pytest.mark.parametrize("M,N,K,name", [
    (1, 14336, 4096, "ROWS"), (3, 3829, 3984, "ROWS"), (65, 12001, 4096, "TILE64"), (257, 4097, 4096, "TILE64"),
    (777, 5002, 4112, "TILE128"), (6449, 1003, 1040, "TILE128"), (16384, 14336, 4096, "TILE256"), (8000, 12000, 9600, "TILE256"),
])
def test_dense(M, N, K, name):
    m = _mx()
    assert m.dense_variant(INT8, INT8, 0, M, N, K) == getattr(m, "DENSE_" + name)


@pytest.mark.parametrize("G,M,N,K,name", [
    (8, 1, 14336, 4096, "ROWS"), (8, 128, 4608, 7168, "STREAM64"), (33, 1024, 2048, 4096, "STREAM64"),
    (256, 16384, 1024, 512, "STREAM128"), (8, 1024, 4608, 7168, "STREAM128"), (2, 9170, 9184, 4096, "TILED"),
    (8, 16384, 4608, 7168, "TILED"),
])
def test_grouped(G, M, N, K, name):
    m = _mx()
    assert m.grouped_int8_variant(G, M, N, K) == getattr(m, "GROUPED_" + name)


@pytest.mark.parametrize("G,N,K", [(8, 14336, 4096), (8, 28672, 4096), (16, 28672, 4096), (64, 1536, 4096), (64, 2816, 2048),
                                   (128, 1536, 4096), (160, 2048, 5120), (256, 4096, 7168), (256, 7168, 2048), (512, 768, 2048)])
def test_few_rows_per_group_take_no_tiles_of_256_rows(G, N, K):
    """Every group that owns rows takes a row tile of its own, and no kernel
    reads its weights faster than the memory does: 1 to 30 rows a group."""
    m = _mx()
    for per in (1, 2, 4, 8, 16, 30):
        for rows in (G * per - 1, G * per, G * per // 2 + 1):
            assert m.grouped_int8_variant(G, rows, N, K) != m.GROUPED_TILED, rows
