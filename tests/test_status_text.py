"""Messages of statuses that several calls return (no GPU needed)."""
from attention_fa2_forward_02_gb300 import binding
from attention_fa2_forward_02_gb300 import build as build_mod


def test_the_workspace_status_names_both_sizes():
    build_mod.build()
    text = binding.library().fa2_status_string(6).decode()
    assert "fa2_backward_workspace_size" in text and "fa2_decode_workspace_size" in text
