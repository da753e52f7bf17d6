"""The 8-bit product's planner on the CPU (256 compute units): its picks held
against measured times, and the shapes of the GPU tests against all it picks."""
import random

import pytest

import lora_bypass_linear_amd as L

NAME = {256: "L", 128: "M", 64: "S"}

# us of a whole call by (tile, K split), MI355X: the picks worth taking and the
# neighbours a wrong model falls for
MEASURED = [
    ((64, 4096, 4096, L.BF16), {"S4": 12.0, "M4": 13.1, "S2": 13.9, "S8": 14.2, "M1": 18.9, "S1": 17.6, "L8": 18.4}),
    ((64, 4096, 4096, L.F32), {"S4": 13.5, "S8": 15.5, "M8": 16.7, "S2": 16.8, "S1": 23.0, "M1": 38.1}),
    ((96, 5120, 5120, L.BF16), {"M4": 16.0, "M2": 18.7, "S2": 19.9, "S4": 20.8, "S1": 21.6, "L8": 21.8, "M1": 22.7}),
    ((96, 5120, 5120, L.F32), {"M4": 22.0, "S4": 24.7, "S2": 26.0, "S1": 28.1, "M2": 30.9, "L8": 30.5}),
    ((128, 1024, 8192, L.BF16), {"S8": 12.9, "S4": 14.4, "M8": 14.6, "M4": 16.4, "S1": 31.2, "M1": 33.0}),
    ((256, 2048, 4096, L.BF16), {"S4": 13.2, "M4": 13.5, "M8": 13.9, "S2": 14.2, "M2": 16.1, "S1": 18.0, "M1": 19.1}),
    ((256, 2048, 4096, L.F32), {"S4": 15.8, "M8": 16.6, "S2": 17.2, "M4": 18.9, "S1": 23.3, "M1": 39.1}),
    ((300, 1040, 2064, L.F32), {"S4": 12.9, "S2": 13.1, "S1": 14.2, "M4": 16.4, "S8": 17.0}),
    ((777, 4096, 4096, L.BF16), {"M1": 21.6, "M2": 34.9, "S1": 40.5, "L2": 42.8, "L1": 47.8}),
    ((1024, 1024, 8192, L.BF16), {"M4": 22.5, "M2": 26.4, "S2": 27.6, "S1": 32.0, "M1": 33.2, "L8": 33.4}),
    ((1024, 1024, 8192, L.F32), {"M4": 32.3, "S2": 37.6, "S4": 40.1, "S1": 42.2, "M2": 45.7, "L8": 48.5}),
    ((2048, 1024, 8192, L.F32), {"M2": 50.5, "M4": 56.3, "S1": 58.2, "S2": 65.2, "L4": 73.1, "M1": 74.5}),
    ((2048, 2048, 8192, L.BF16), {"M1": 39.7, "M2": 54.4, "L2": 64.3, "S1": 74.1, "L1": 87.5}),
    ((2500, 2500, 2512, L.BF16), {"M1": 41.6, "L1": 50.9, "S1": 57.7}),
    ((2560, 2560, 2560, L.BF16), {"M1": 29.4, "L1": 34.3, "S1": 50.0}),
    ((4096, 4096, 4096, L.BF16), {"L1": 69.0, "M1": 91.4, "S1": 153.7}),
    ((16384, 8192, 1024, L.F32), {"L1": 317.2, "M1": 412.7, "S1": 538.2}),
]


@pytest.mark.parametrize("case,us", MEASURED)
def test_pick_is_near_the_best_measured(case, us):
    tn, _, ks = L.fp8_linear_plan(*case)
    assert us[NAME[tn] + str(ks)] <= 1.1 * min(us.values())


def test_workspace_covers_every_output_dtype():
    rng = random.Random(3)
    for _ in range(2000):
        M, N, K = int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(4, 13)), 16 * int(2 ** rng.uniform(0, 9))
        need = L.fp8_linear_workspace_size(M, N, K)
        for dt in (L.F16, L.BF16, L.F32):
            ks = L.fp8_linear_plan(M, N, K, dt)[2]
            assert ks == 1 or need >= ks * M * N * 4, (M, N, K, dt)


def test_few_rows_and_empty():
    assert L.fp8_linear_plan(1, 4096, 4096, L.BF16) == (16, 16, 1)
    assert L.fp8_linear_plan(32, 8192, 4096, L.F32) == (32, 32, 1)
    assert L.fp8_linear_plan(0, 64, 64, L.BF16) == (0, 0, 1)


def test_refusals():
    for bad in ((-1, 16, 16, 2), (4, 16, 16, 0), (4, 16, 24, 2)):
        with pytest.raises(L.LycError):
            L.fp8_linear_plan(*bad)
    assert L.lib().lyc_fp8_linear_plan(64, 64, 64, 2, None, None, None) == L.OK


def _path(M, N, K, dt):
    tn, _, ks = L.fp8_linear_plan(M, N, K, dt)
    blocks = -(-K // 128)
    return tn, ks > 1, dt == L.F32, ks > 1 and -(-blocks // ks) * (ks - 1) >= blocks


def test_gpu_shapes_reach_every_path():
    """(tile, split, widened sums, last split empty) of 20000 shapes of more
    than 32 rows: each is taken by the GPU tests, with and without the fold."""
    from tests.test_gpu_fp8_paths import CASES, F32, RAGGED
    with_fold = {_path(M, N, K, L.F32 if F32 in (dt, adt) else L.BF16) for M, N, K, _, dt, adt in CASES}
    by_element = {_path(M, N, K, L.dtype_code(out))[:2] for M, N, K, out in RAGGED}
    assert by_element == {(256, False), (256, True), (128, False), (128, True), (64, False), (64, True)}
    rng = random.Random(7)
    for _ in range(10000):
        M, N, K = int(33 * 2 ** rng.uniform(0, 8)), 16 * int(2 ** rng.uniform(0, 9)), 16 * int(2 ** rng.uniform(0, 9.2))
        for dt in (L.BF16, L.F32):
            assert _path(M, N, K, dt) in with_fold, (M, N, K, dt, _path(M, N, K, dt))
