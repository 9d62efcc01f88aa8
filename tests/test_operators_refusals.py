"""What the attention entry points refuse beyond their sizes (on the host, before any HIP call)."""

import os

import pytest

from gated_delta_rule_kla_amd import kla

pytestmark = pytest.mark.skipif(not os.path.exists(kla.lib_path()), reason="libkla.so not built")

FAKE = 0x7F0000000000  # never dereferenced
PARAM, NULL, WORKSPACE = -11, -1, -7


def prompts(scale, q=FAKE):
    return kla.lib().kla_attn_fwd(q, FAKE, FAKE, scale, FAKE, FAKE, None, None, None, None, 2, 2, 8, 4, 10, 10, 128, 0,
                                  None)


def token(scale, q=FAKE):
    return kla.lib().kla_attn_kv4_decode_step(q, FAKE, FAKE, FAKE, FAKE, scale, FAKE, 2, 8, 4, 128, 8, 16, 4, 64, 0,
                                              None, 0, None)


@pytest.mark.parametrize("call", [prompts, token])
@pytest.mark.parametrize("scale", [3.4e38, -3.4e38, 2.4e38, float("nan"), float("inf"), -float("inf")])
def test_scales_beyond_fp32_in_base_two(call, scale):
    """The kernels take scale log2(e), which has to be finite too: 2.36e38 is where it is not."""
    assert call(scale) == PARAM


@pytest.mark.parametrize("call", [prompts, token])
@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 0.0, 1e-45])
def test_scales_that_are_taken(call, scale):
    assert call(scale, q=None) == NULL  # past the scale's check


def test_a_missing_workspace_names_no_other_operators_function():
    """The status is shared: its text must not send a caller of the recurrence or of the decode step
    to kla_chunk_workspace_bytes."""
    lib = kla.lib()
    st = lib.kla_attn_kv4_decode_step(FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, 2, 8, 4, 128, 8, 16, 10000, 100000, 0,
                                      None, 0, None)
    assert st == WORKSPACE
    text = lib.kla_status_str(st).decode()
    assert "workspace" in text and "kla_chunk" not in text
