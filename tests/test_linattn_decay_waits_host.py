"""Options of the decayed attention's calls (no GPU needed)."""
import pytest

from test_linattn_decay_host import F, INVALID, W, view  # noqa: F401  (W: the fixture)


@pytest.mark.parametrize("options,code", [(dict(kernel=1), INVALID), (dict(kernel=-1), INVALID),
                                          (dict(spin_limit=-1), INVALID), (dict(spin_limit=5), 0), (None, 0)])
def test_options(W, options, code):  # noqa: F811
    """Refused before any launch; T = 0 does nothing else."""
    opt = None if options is None else W.abi.Options(**options)
    v = [view(W, i + 1) for i in range(7)]
    assert W.abi.linattn_decay_forward_ex(1, 0, 2, 32, 32, 0, *v[:3], F, 1.0, 0, 0, v[3], 0, 0, 0, 0, 0, opt) == code
    assert W.abi.linattn_decay_backward_ex(1, 0, 2, 32, 32, 0, *v[:3], F, 1.0, 0, 0, v[3], 0, *v[4:], 0, 0, 0, 0, 0,
                                           opt) == code


def test_status_word_needs_a_place(W):  # noqa: F811
    assert W.abi.lib.linattn_decay_status_word(None) == INVALID
