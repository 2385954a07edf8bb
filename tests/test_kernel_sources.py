"""What every kernel's source keeps to (no GPU)."""
import os
import re

from activation_epilogue_gb300 import build as libbuild


def test_no_non_coherent_loads():
    """The kernels start while their stream's previous work still runs (programmatic dependent launch) and
    read what it writes.  Loads through the read-only path are for memory that no one writes during the
    kernel's whole life, the part before its wait included: they are not used."""
    found = []
    for name in sorted(os.listdir(libbuild.CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(libbuild.CSRC, name)) as fh:
                for i, line in enumerate(fh, 1):
                    if re.search(r"__ldg\s*\(|ld\.global[\w.]*\.nc\b", line):
                        found.append(f"{name}:{i}")
    assert not found, found
