"""What the wrappers around the experts give back, on the stand-ins of test_layer_machine_host
(no GPU needed)."""
import pytest

from tests.test_layer_machine_host import F32, col, machine, x  # noqa: F401


@pytest.mark.parametrize("block", [False, True])
def test_the_norms_give_back_only_what_they_write(machine, block):  # noqa: F811
    """Without w_next there is no n, whatever pair of outputs is given; without a block out is x."""
    g, log, _ = machine
    here, o, n = x(F32), x(F32), x()
    if block:
        assert g.norm_join(here, x(), col(), out=(o, n)) == (o, None)
        assert g.norm_join(here, x(), col(), out=(o, None)) == (o, None)
        assert g.norm_join(here, x(), col(), w_next=col(), out=(o, n)) == (o, n)
    else:
        assert g.norm_join(here, w_next=col(), out=(o, n)) == (here, n)
        assert g.norm_join(here, w_next=col(), out=(None, n)) == (here, n)
