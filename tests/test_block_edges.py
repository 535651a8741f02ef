"""What the header says of the block norm's, the selective scan's and the short convolution's arguments, by the host-side checks."""
import os
import re

import pytest

from test_block_abi import NULL, OK, norm_desc, norm_fwd
from test_sequence_layer_amd import profiling


def test_norm_parameters_without_an_output():
    assert norm_fwd(norm_desc(), y=None) == OK                       # gamma_pre and beta_pre reach nothing
    assert norm_fwd(norm_desc(), y=None, bn=None) == OK
    assert norm_fwd(norm_desc(), y=None, gn=None, bn=None) == OK
    assert norm_fwd(norm_desc(), gn=None) == NULL and norm_fwd(norm_desc(), gn=None, bn=None) == NULL
    assert norm_fwd(norm_desc(), y=None, gn=None) == NULL            # beta_pre alone
    assert norm_fwd(norm_desc(), s=None, y=None) == NULL


def included(path, seen):
    for name in re.findall(r'#include "([^"/]+)"', open(path).read()):
        if name not in seen:
            seen.add(name)
            included(os.path.join(os.path.dirname(path), name), seen)
    return seen


@pytest.mark.parametrize("source", ["scan_fwd.hip", "scan_bwd.hip", "short_conv.hip", "block_norm.hip", "block_sum.hip"])
def test_profiles_know_the_kernels_sources(source):
    """A profile record is tied to every file that its kernel is made of."""
    path = os.path.join(profiling.PKG, "csrc", source)
    kernels = re.findall(r"__global__[^;{]*?void (ttt_\w+)\(", open(path).read())
    assert kernels
    for k in kernels:
        assert set(profiling.KERNEL_SOURCES[k]) == {source} | included(path, set()), k
