"""The launches of the products grouped by expert over the whole range of sizes that the C ABI takes, from the library's
own rules, without a GPU: every index that a kernel makes of its launch stays where it belongs."""
import itertools

import pytest

import grouped_plan as plan

POSITIONS, DIM, OUT, EXPERTS = 1 << 23, 65536, 1 << 37, 512
SIZES = [(E, P, N) for E, P, N in itertools.product(
    (1, 2, 3, 60, 256, 511, 512),
    (1, 2, 63, 64, 65, 129, 1000, 16384, 131071, 1 << 19, 1 << 20, (1 << 20) + 1, 1 << 21, (1 << 22) - 1, 1 << 22, POSITIONS - 1, POSITIONS),
    (1, 8, 129, 257, 2040, 2048, 4096, 8184, 8192, 8200, 16384, 32768, 65528, DIM)) if P * N <= OUT]


def launches(E, P, N):
    f = plan.forward(True, E, P, N)
    if f != "few":
        yield "product", f, True
    yield "rows' gradient", plan.turned(E, P, N), True


def test_tiled_launches_hold_their_tiles():
    for E, P, N in SIZES:
        for what, form, ragged in launches(E, P, N):
            groups = plan.workgroups(form, ragged, E, P, N)
            assert groups >= plan.row_tiles(form, ragged, E, P) * plan.col_tiles(form, N), (what, E, P, N)
            assert groups * form[0] * 64 < 1 << 32, (what, form, E, P, N)  # threads of a launch


def test_what_a_kernel_counts_in_32_bits():
    """The tiles' numbers times the column tiles, also of offsets that do not ascend: every second expert may have all rows."""
    for E, P, N in SIZES:
        for what, form, ragged in launches(E, P, N):
            tiles = (E + 1) // 2 * (P // form_lowest(form) + 1) + E + 2
            assert tiles * plan.col_tiles(form, N) < 1 << 31, (what, form, E, P, N)


def form_lowest(form):
    waves, height = form
    return height or (128 if waves == 8 else 64)


def test_dense_launches():
    """All rows one group, up to 2^24 of them (8-bit products)."""
    for M, N in itertools.product((65, 100, 4097, 1 << 20, 1 << 24), (1, 17, 4096, 8192, 65537, 1 << 20, 1 << 24)):
        form = plan.forward(False, 1, M, N)
        if M * N <= OUT:
            groups = plan.workgroups(form, False, 1, M, N)
            assert groups >= -(-M // form_lowest(form)) * plan.col_tiles(form, N) and groups * form[0] * 64 < 1 << 32
            assert groups < 1 << 31


def test_weights_gradient_launches():
    for E, N, K in itertools.product((1, 3, 32, 60, 256, 512), (8, 120, 136, 1032, 4096, 16384, 65528, DIM), (8, 72, 264, 1000, 4104, 16384, DIM)):
        if E * N * K <= OUT:
            if plan.dw_large(E, N, K):
                assert plan.dw_workgroups(True, E, N, K) * 512 < 1 << 32
            assert plan.dw_workgroups(False, E, N, K) * 256 < 1 << 32  # rows far apart take these at any size


@pytest.mark.parametrize("P,N", [(1 << 20, 65536), (POSITIONS, 8192), (POSITIONS, 16384)])
def test_results_of_128_gib_and_more(P, N):
    """2^36 and 2^37 values in rows of one expert: a launch whose threads have numbers below 2^31 or counts them in 64 bits;
    four waves' tiles were 2^23, 256 threads each, and more."""
    form = plan.turned(1, P, N)
    assert form == (8, 128) and plan.workgroups((4, 64), True, 1, P, N) * 256 > 1 << 31
    assert plan.workgroups(form, True, 1, P, N) * 512 < 1 << 32
