"""Refusals of the operators with scales of 128 that need no GPU."""
import pytest

from mxfp8_block_scaled_mxgemm_amd import _block


@pytest.mark.parametrize("table,what", [(_block._PRECISION, "precision mode"), (_block.SCORES, "score"),
                                        (_block.NORMS, "norm")])
@pytest.mark.parametrize("name", ["fast", None, 7, ["exact"]])
def test_unknown_choices_are_value_errors_that_name_the_known_ones(table, what, name):
    with pytest.raises(ValueError, match=f"unknown {what} .*: one of {next(iter(table))}, "):
        _block._pick(table, name, what)
