"""Which kernels a backward pass of the experts takes, on both sides of each bound
(no GPU): sizes that were measured with either. The one kernel's time, the two
kernels', in us on a GB300."""
import pytest

import tuning_reference as tune

# rows, experts, n, k
ONE = [(1024, 64, 1024, 512),  # 33 and 36
       (66, 66, 1024, 512), (1056, 66, 1024, 512), (4864, 76, 1024, 512),  # 31.6 and 33.3, 33.4 and 36.7, 40.7 and 46.2
       (1216, 76, 512, 1024),  # 37.6 and 40.9
       (1536, 16, 512, 1024), (4096, 16, 512, 512),  # 15.8 and 20.5, 15.2 and 19.3
       (24576, 256, 256, 256),  # 33.1 and 52.7
       (9216, 96, 512, 512),  # 33.3 and 39.6
       (300, 4, 512, 512), (1001, 5, 513, 1001),
       (1024, 1, 64, 64), (1536, 1, 64, 64), (2048, 1, 16, 64)]  # 8.9 and 11.6, 10.7 and 13.3, 12.7 and 15.2
TWO = [(4, 1, 4096, 4096), (16, 4, 4096, 1024), (20, 4, 4096, 2304),  # a long dx: 32.2 and 28.0, 31.7 and 28.0, 43 and 39
       (8192, 16, 64, 4096), (2048, 2, 64, 4096),  # a wide dx: 60.0 and 38.0, 24.3 and 18.7
       (4096, 4, 4096, 4096),
       (32768, 64, 1024, 512),  # many rows
       (64, 8, 4096, 4096), (2, 8, 14336, 4096),  # large weights: 107 and 103, 249 and 210
       (65536, 16, 96, 200), (8192, 1, 128, 128)]  # long sums: 72.9 and 34.1


@pytest.mark.parametrize("shape", ONE + TWO, ids=str)
def test_one_kernel_or_two(shape):
    kinds = [q["kind"] for q in tune.grouped_plan(*shape, True) if q["kind"] in ("mode", "both")]
    assert kinds == (["both"] if shape in ONE else ["mode", "mode"])


@pytest.mark.parametrize("n,k", [(256, 256), (512, 512), (1024, 512), (512, 1024), (1024, 1024)])
def test_a_few_more_experts_or_rows_go_the_same_way(n, k):
    """Whatever their number, up to and past 2^25 weights."""
    for experts in range(1, (1 << 25) // (n * k) + 3):
        for rows in (experts, 15 * experts, 47 * experts):
            assert tune.grouped_plan(rows, experts, n, k, True)[0]["kind"] == "both", (rows, experts)


# whether dW's sums are taken in parts and joined
WHOLE = [(3000, 1, 256, 256), (6000, 2, 128, 128), (12000, 4, 64, 64)]  # 21.1 and 30.9, 20.6 and 29.1, 21.4 and 30.2
PARTS = [(16384, 2, 128, 1024), (32768, 4, 256, 256), (8192, 1, 64, 64)]  # 50.8 and 35.5, 51.3 and 31.5, 34.8 and 25.9


@pytest.mark.parametrize("shape", WHOLE + PARTS, ids=str)
def test_sums_whole_or_in_parts(shape):
    dw, = [q for q in tune.grouped_plan(*shape, True) if q["kind"] == "mode" and q["mode"] == 2]
    assert dw["split"] == (shape in PARTS)
