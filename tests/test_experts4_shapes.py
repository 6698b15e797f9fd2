"""The products that the GPU tests make, by the kernel and the groups of a slab that they take."""
import itertools

from tests import product4_shapes as S

KERNELS, GROUPS = ("narrow", "middle", "stream", "square", "wide"), (4, 2, 1)


def taken(T, M, E, N, H, group):
    return S.kernel_of(M, E, N, H), S.groups_of_a_slab(group)


def test_streamed_products_take_every_streamed_kernel_past_two_slabs_for_a_wave():
    even, odd = set(), set()
    for kernel, shapes in S.LONG.items():
        for T, M, E, N, H in shapes:
            assert S.kernel_of(M, E, N, H) == kernel and H % 128
    for case in S.STREAMED:
        kernel, parts = taken(*case)
        most = max(S.slabs_of_waves(kernel, case[4]))
        assert most >= 3
        (odd if most % 2 else even).add((kernel, parts))
    every = set(itertools.product(("narrow", "middle", "stream"), GROUPS))
    assert odd == every and even == every


def test_part_slabs_come_to_every_kernel():
    assert {taken(*case) for case in S.PART_SLABS} == set(itertools.product(KERNELS, (4, 2)))
    for _, _, _, _, H, group in S.PART_SLABS:
        assert -(-(H % 128) // group) < 128 // group     # groups that the last slab lacks


def test_every_kernel_is_tested():
    from tests.test_gpu_experts4 import MANY, PRODUCTS
    cases = PRODUCTS + MANY + S.STREAMED + S.PART_SLABS
    assert {taken(*case) for case in cases} == set(itertools.product(KERNELS, GROUPS))
