"""What the header says of the block norm's, the selective scan's and the short convolution's arguments, by the host-side checks."""
from test_block_abi import NULL, OK, norm_desc, norm_fwd


def test_norm_parameters_without_an_output():
    assert norm_fwd(norm_desc(), y=None) == OK                       # gamma_pre and beta_pre reach nothing
    assert norm_fwd(norm_desc(), y=None, bn=None) == OK
    assert norm_fwd(norm_desc(), y=None, gn=None, bn=None) == OK
    assert norm_fwd(norm_desc(), gn=None) == NULL and norm_fwd(norm_desc(), gn=None, bn=None) == NULL
    assert norm_fwd(norm_desc(), y=None, gn=None) == NULL            # beta_pre alone
    assert norm_fwd(norm_desc(), s=None, y=None) == NULL
