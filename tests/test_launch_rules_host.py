"""The launch rules go by the device's own number of SMs."""
import os
import re

import sparse_attention_top_gb300 as gb

CSRC = os.path.join(os.path.dirname(gb.__file__), "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_rule_names_one_gpus_number_of_sms():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            assert not re.search(r"\b1(44|48|52)\b", code(name)), name


def test_the_size_of_a_workspace_needs_no_device():
    assert gb.gbtopk_verify_workspace_bytes(64, 131073, 16) > 0
    assert gb.gbtopk_attention_workspace_bytes(64, 32, 8, 128) > 0
