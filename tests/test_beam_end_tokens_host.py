"""End tokens that do not fit into 32 bits are refused, not cut to another token."""
import pytest

from test_kv_share_binding_host import _beam, calls, refused  # noqa: F401


@pytest.mark.parametrize("tokens", [[5 + (1 << 32)], [1, 1 << 31], (-(1 << 31) - 1,), [1 << 40, 2]])
def test_wide_end_tokens(calls, tokens):  # noqa: F811
    refused(lambda: _beam(end_tokens=tokens), calls)


@pytest.mark.parametrize("tokens", [[], (), [7], (7, 8), [(1 << 31) - 1, -1]])
def test_others_are_taken(calls, tokens):  # noqa: F811
    _beam(end_tokens=tokens)
    assert calls == ["wsw_beam_select"]
