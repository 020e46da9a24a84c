"""The gated recurrence's kernels hold no divergent branch in their loops over tiles.

The compiler has been seen to place copies of live registers at the join of such a
branch before it restores the execution mask, so that lanes that did not take it went on with
stale addresses.  The loops are written without any (range checks, selects and
uniform votes in their place); this looks for the execution mask being written inside
a loop in the listings that the build's own flags give, so that a later edit or
compiler that brings a branch back is found without a GPU."""

import concurrent.futures
import os
import re
import subprocess

from selective_state_space_23_amd import build

WRITES_EXEC = re.compile(r"\bs_\w+\s+exec(_lo|_hi)?\b|_saveexec_|\bv_cmpx_")


def loops(listing):
    """{kernel: [instructions in its loops that write the execution mask]} of the kernels with loops."""
    found, kernel, inside = {}, None, False
    for line in listing.splitlines():
        if m := re.match(r"(_Z\w+):", line):
            kernel, inside = m.group(1), False
        elif re.match(r"\.LBB\w+:|; %bb\.\d+:", line):
            inside = "Loop" in line
        elif re.match(r"\s+;.*Loop", line):   # a block whose note goes on over more lines
            inside = True
        text = line.split(";")[0].strip()
        if inside and text and not text.startswith(".") and not text.endswith(":"):
            hits = found.setdefault(kernel, [])
            if WRITES_EXEC.search(text):
                hits.append(text)
    return found


def test_the_search_finds_a_divergent_loop():
    listing = """
_Z6kernelPf:                            ; @_Z6kernelPf
; %bb.0:
	s_and_saveexec_b64 s[0:1], vcc
.LBB0_1:                                ; =>This Loop Header: Depth=1
                                        ;     Child Loop BB0_2 Depth 2
	v_add_f32_e32 v0, v1, v2
.LBB0_2:                                ;   Parent Loop BB0_1 Depth=1
                                        ; =>  This Inner Loop Header: Depth=2
	s_and_saveexec_b64 s[2:3], vcc
; %bb.3:                                ;   in Loop: Header=BB0_2 Depth=2
	s_or_b64 exec, exec, s[2:3]
; %bb.4:
	s_or_b64 exec, exec, s[0:1]
_Z5otherPf:                             ; @_Z5otherPf
	s_mov_b64 exec, s[0:1]
"""
    assert loops(listing) == {"_Z6kernelPf": ["s_and_saveexec_b64 s[2:3], vcc", "s_or_b64 exec, exec, s[2:3]"]}


def test_no_divergent_branch_in_the_loops_over_tiles(tmp_path):
    def listing(name):
        out = str(tmp_path / (name + ".s"))
        cmd = build.compile_cmd(os.path.join(build.CSRC, name + ".hip"), out)
        cmd[cmd.index("-c")] = "-S"
        r = subprocess.run(cmd[:1] + ["--cuda-device-only"] + cmd[1:], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        with open(out) as f:
            return f.read()

    with concurrent.futures.ThreadPoolExecutor() as pool:
        texts = list(pool.map(listing, ("recurrence", "recurrence_bwd")))
    for text, name in zip(texts, ("rec_fwd_kernel", "rec_bwd_kernel")):
        kernels = {m for m in re.findall(r"^(_Z\w+):", text, re.M) if name in m}
        found = {k: v for k, v in loops(text).items() if name in k}
        assert kernels and set(found) == kernels, "every kernel has its loop over tiles"
        bad = {k: v for k, v in found.items() if v}
        assert not bad, bad
