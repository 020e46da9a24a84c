"""The gated delta rule's kernels and those of the head norms hold no divergent branch in their loops
(tests/test_kernel_listings.py tells why, and has the search)."""

import os
import re
import subprocess

import pytest

from selective_state_space_23_amd import build
from test_kernel_listings import loops


@pytest.mark.parametrize("source,names", [
    ("delta_fwd", ("fwd_kernel", "fwd_pairs_kernel")),
    ("delta_bwd", ("bwd_states_kernel", "bwd_pairs_kernel")),
    ("delta_grads", ("grads_kernel",)),
    ("qk_norm", ("norm_kernel",)),
])
def test_no_divergent_branch_in_the_loops(tmp_path, source, names):
    out = str(tmp_path / (source + ".s"))
    cmd = build.compile_cmd(os.path.join(build.CSRC, source + ".hip"), out)
    cmd[cmd.index("-c")] = "-S"
    r = subprocess.run(cmd[:1] + ["--cuda-device-only"] + cmd[1:], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    with open(out) as f:
        text = f.read()
    for name in names:
        kernels = {m for m in re.findall(r"^(_Z\w+):", text, re.M) if re.search(r"\d" + name + "I", m)}
        found = {k: v for k, v in loops(text).items() if k in kernels}
        assert kernels and set(found) == kernels, (name, "every kernel has its loop")
        bad = {k: v for k, v in found.items() if v}
        assert not bad, bad
