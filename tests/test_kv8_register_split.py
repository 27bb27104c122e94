"""setmaxnreg is defined only where every warp of a warpgroup executes the same one: each stands first in a branch whose
condition cuts at whole warpgroups (four warps)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_decode_attention_03_gb300", "csrc")


def branches_of_splits(text):
    """The condition of the branch that each regs_inc / regs_dec stands first in."""
    lines = [line for line in text.splitlines() if line.strip() and not line.strip().startswith("//")]
    for at, line in enumerate(lines):
        if re.match(r"\s*regs_(inc|dec)<\d+>\(\);", line):
            yield lines[at - 1].strip()


@pytest.mark.parametrize("name", ["mla_decode_kv8.cu", "mla_decode_kv8_pair.cu"])
def test_register_splits_cut_at_whole_warpgroups(name):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    values = {k: int(v) for k, v in re.findall(r"constexpr int (k\w+) = (\d+);", text)}
    found = list(branches_of_splits(text))
    assert len(found) >= 2
    for branch in found:
        if branch == "} else {":
            continue
        warps = re.fullmatch(r"(?:\} else )?if \(warp < ([\w +]+)\) \{", branch)
        assert warps, f"{name}: a split of registers inside `{branch}`"
        assert sum(values[t] if t in values else int(t) for t in warps.group(1).split(" + ")) % 4 == 0, branch
