"""What the sources of the compiled library must not hold, read as text (no GPU)."""

import glob
import os
import re

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "fsdp_sharded_optimizer_flatparameter_gb300", "csrc", "*")))


def _instructions(text, name):
    """Inline assembly instructions that begin with `name`, their string literals joined."""
    joined = re.sub(r'"\s*"', "", text)
    return re.findall(re.escape(name) + r'[^;"]*', joined)


def test_no_copy_is_multicast():
    """The library is loaded by one process per GPU too (ZeroRank): its copies write their own CTA's shared memory only."""
    seen = 0
    for path in SOURCES:
        with open(path) as f:
            for line in _instructions(f.read(), "cp.async.bulk"):
                seen += 1
                assert "multicast" not in line, "%s: %s" % (os.path.basename(path), line)
    assert seen >= 3


def test_what_calls_remember_is_safe_between_threads():
    """Calls may come from several threads: what the 8-bit operators' host code keeps between calls is constant or atomic."""
    for path in SOURCES:
        if not os.path.basename(path).startswith("q8"):
            continue
        with open(path) as f:
            for n, line in enumerate(f, 1):
                if re.match(r"\s*static ", line):
                    assert re.match(r"\s*static (const\b|constexpr\b|std::atomic<)", line), "%s:%d: %s" % (path, n, line)
