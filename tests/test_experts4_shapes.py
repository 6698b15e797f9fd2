"""The products that the GPU tests make, by the kernel and the groups of a slab that they take."""
import itertools

from tests import product4_shapes as S

KERNELS, GROUPS = ("narrow", "middle", "stream", "square", "wide"), (4, 2, 1)


def taken(T, M, E, N, H, group):
    return S.kernel_of(M, E, N, H), S.groups_of_a_slab(group)


def test_part_slabs_come_to_every_kernel():
    assert {taken(*case) for case in S.PART_SLABS} == set(itertools.product(KERNELS, (4, 2)))
    for _, _, _, _, H, group in S.PART_SLABS:
        assert -(-(H % 128) // group) < 128 // group     # groups that the last slab lacks
